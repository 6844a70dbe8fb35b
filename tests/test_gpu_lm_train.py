"""The language-model operators together: the training example, and its gradients against a plain model."""
import math
import os
import sys

import pytest
import torch

from tests.helpers import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_learns(bits):
    """A uniform guess costs log 64; the permutation can be learnt, so that the loss falls below half of it."""
    import train_step
    say(f"[lm] training example, {bits}-bit moments")
    losses = train_step.train(steps=120, vocab=64, d=256, layers=2, rows=4, length=64, bits=bits, report=0)
    assert all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(64)) < 1.0
    assert sum(losses[-10:]) / 10 < 0.5 * math.log(64), losses[-10:]


def test_gradients_of_the_model():
    """The head's and the norms' part of the model (no mixer) against a plain FP32 model: BF16 streams, so within a few
    roundings of 2^-8 in the L2 sense."""
    from linear_recurrence_sequence_amd import autograd
    say("[lm] norms and head against torch")
    g = torch.Generator(device="cuda").manual_seed(1)
    n, d, v = 200, 64, 300

    def r(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    x, y, gate, w = r(n, d), r(n, d).bfloat16(), r(n, d).bfloat16(), r(v, d, std=d ** -0.5).bfloat16()
    vec = [1.0 + r(d, std=0.1) for _ in range(3)]
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[::7] = -1

    def leaves():
        return [a.clone().requires_grad_() for a in (x, y, gate, *vec, w)]

    ours = leaves()
    out, h = autograd.block_norm(ours[0], ours[1], ours[2], ours[3], ours[4], ours[5], gate_act="silu")
    loss, lse = autograd.linear_ce(h, ours[6], t, softcap=20.0)
    (loss.sum() / n + 1e-3 * (lse * lse).mean() + (out * out).mean()).backward()
    theirs = [a.float().detach().requires_grad_() for a in leaves()]
    a, b, c, w1, sc, w2, wf = theirs

    def norm(z, k):
        return z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * k

    s = a + sc * torch.nn.functional.silu(c) * norm(b, w1)
    z = norm(s, w2) @ wf.t()
    z = 20.0 * torch.tanh(z / 20.0)
    e = torch.logsumexp(z, 1)
    on = t >= 0
    ce = torch.where(on, e - z.gather(1, t.clamp_min(0)[:, None])[:, 0], torch.zeros_like(e))
    (ce.sum() / n + 1e-3 * (e * e).mean() + (s * s).mean()).backward()
    for name, p, q in zip(("x", "y", "gate", "w_post", "scale", "w_pre", "w"), ours, theirs):
        err = float((p.grad.float() - q.grad).norm() / q.grad.norm())
        assert err < 4 * 2.0 ** -8, (name, err)


def test_a_stream_given_owns_what_the_call_allocates():
    """Results on a stream that is not current, while the current one keeps reusing the memory it frees."""
    from linear_recurrence_sequence_amd import lm
    say("[lm] a stream given")
    g = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(300, 64, generator=g, device="cuda").bfloat16()
    w = torch.randn(5000, 64, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, 5000, (300,), generator=g, device="cuda")
    x, k = torch.randn(300, 64, generator=g, device="cuda"), torch.ones(64, device="cuda")
    loss, lse = lm.linear_ce_fwd(h, w, t)
    want = lm.linear_ce_bwd(h, w, t, lse, loss)
    r, n, stats = lm.block_norm_fwd(x, x, None, k, k, k)
    gn = lm.block_norm_bwd(x, x, None, k, k, k, stats, r, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        l2, e2 = lm.linear_ce_fwd(h, w, t, stream=side)
        got = lm.linear_ce_bwd(h, w, t, lse, loss, stream=side)
        r2, n2, s2 = lm.block_norm_fwd(x, x, None, k, k, k, stream=side)
        gn2 = lm.block_norm_bwd(x, x, None, k, k, k, stats, r, n, stream=side)
        torch.full((1 << 20,), float("nan"), device="cuda")
        side.synchronize()
        assert torch.equal(l2, loss) and torch.equal(e2, lse) and torch.equal(r2, r) and torch.equal(n2, n)
        assert all(torch.equal(got[a], want[a]) for a in want) and all(torch.equal(gn2[a], gn[a]) for a in gn)
