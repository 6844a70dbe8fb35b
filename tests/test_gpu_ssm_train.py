"""The selective scan, the convolution and the embedding together, as a model uses them: the training example, its
gradients, prompts and then single tokens, and other devices."""
import math
import os
import sys

import pytest
import torch

from linear_recurrence_sequence_amd import lm, ssm
from tests.helpers import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def test_the_example_runs():
    import train_step
    say("[ssm] training example")
    losses = train_step.train(steps=4, vocab=64, d=96, layers=2, rows=3, length=50, report=0, mixer="ssm")
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)


def plain_loss(model, tokens, targets):
    """The example's model of state space blocks in torch operations of 64 bits, on the same weights."""
    m = {k: t.detach().double().requires_grad_() for k, t in model.matrices.items()}
    v = {k: t.detach().double().requires_grad_() for k, t in model.vectors.items()}
    d, n, r = model.d, model.states, model.rank

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

    x = m["embed"][tokens]
    h = norm(x, v["norm_in"])
    for i in range(model.layers):
        both = h @ m[f"in{i}"].t()
        branch, w = torch.nn.functional.pad(both[..., :d], (0, 0, 3, 0)), v[f"conv{i}"]
        u = torch.nn.functional.silu(v[f"conv_bias{i}"] + sum(branch[:, k:k + tokens.shape[1]] * w[:, k] for k in range(4)))
        p = u @ m[f"proj{i}"].t()
        s = torch.nn.functional.softplus(p[..., :r] @ m[f"dt{i}"].t() + v[f"dt_bias{i}"])
        rate, state, ys = -torch.exp(v[f"log_rate{i}"]), torch.zeros(tokens.shape[0], d, n, dtype=torch.float64, device="cuda"), []
        for t in range(tokens.shape[1]):
            state = torch.exp(s[:, t, :, None] * rate) * state + (s * u)[:, t, :, None] * p[:, t, None, r:r + n]
            ys.append((state * p[:, t, None, r + n:]).sum(-1) + v[f"skip{i}"] * u[:, t])
        y = torch.stack(ys, 1) * torch.nn.functional.silu(both[..., d:])
        x = x + v[f"scale{i}"] * norm(y, v[f"w_post{i}"])
        h = norm(x, v[f"w_pre{i}"])
    z = 30.0 * torch.tanh(h @ m["embed"].t() / 30.0)
    lse = torch.logsumexp(z, -1)
    on = targets >= 0
    ce = (lse - z.gather(-1, targets.clamp_min(0)[..., None])[..., 0])[on].sum() / on.sum()
    return ce + 1e-4 * (lse * lse).mean(), {**m, **v}


def test_gradients_of_the_model():
    """Every weight's gradient against the same model in 64 bits.  The streams between the operators are BF16: a block rounds about ten times on
    the way forward and as often back, 2^-8 each at most and of either sign; the norms and gates may double that, and two blocks add up: below
    2 sqrt(2 * 2 * 10) 2^-8 = 5% of a gradient's length, where any mistake would be of the order of one."""
    import train_step
    say("[ssm] gradients of the model")
    model = train_step.Model(90, 64, 2, seed=3, mixer="ssm")
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens = torch.randint(0, 90, (2, 40), generator=g, device="cuda")
    targets = torch.randint(0, 90, (2, 40), generator=g, device="cuda")
    targets[0, :5] = -1
    loss, _ = model.loss(tokens, targets)
    loss.backward()
    want, leaves = plain_loss(model, tokens, targets)
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) < 0.02 * float(want.detach())
    for k, t in {**model.matrices, **model.vectors}.items():
        ref = leaves[k].grad
        off = float((t.grad.double() - ref).norm() / ref.norm())
        assert off < 0.05, (k, off)


def test_prompts_then_tokens():
    """Logits after each token, from single steps on what a padded batch of prompts left, against those of the whole rows.  BF16 streams,
    rounded the same way on both sides but where FP32 sums of another order fall on the other side of a tie: within 2^-5 of the
    largest logit."""
    import train_step
    say("[ssm] prompts, then tokens")
    model = train_step.Model(90, 64, 2, seed=4, mixer="ssm")
    g = torch.Generator(device="cuda").manual_seed(6)
    rows, lengths = torch.randint(0, 90, (3, 60), generator=g, device="cuda"), torch.tensor([20, 33, 1], dtype=torch.int32, device="cuda")
    padded = rows[:, :40].clone()
    for i, k in enumerate(lengths.tolist()):
        padded[i, k:] = -1
    logits, states = model.run(padded, lengths=lengths)
    at = lengths.long()
    for _ in range(6):
        for i, k in enumerate(at.tolist()):
            want = model.run(rows[i:i + 1, :k])[0][0]
            assert (logits[i].float() - want.float()).abs().max() <= 2 ** -5 * want.float().abs().max(), (i, k)
        logits, states = model.run(rows.gather(1, at[:, None])[:, 0], states)
        at = at + 1
    out = model.generate(padded, 5, lengths=lengths)
    assert out.shape == (3, 5) and int(out.min()) >= 0 and int(out.max()) < 90


def test_decoding_from_a_graph():
    """A whole step of the model captured and replayed token after token, against the eager one."""
    import train_step
    say("[ssm] decoding from a graph")
    model = train_step.Model(90, 64, 2, seed=7, mixer="ssm")
    prompt = torch.randint(0, 90, (2, 17), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda")
    _, eager = model.run(prompt)
    replayed = [tuple(t.clone() for t in s) for s in eager]
    kept = [tuple(t.clone() for t in s) for s in eager]
    token = torch.zeros(2, dtype=torch.int64, device="cuda")
    model.run(token, [tuple(t.clone() for t in s) for s in eager])            # libraries warm up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, _ = model.run(token, replayed)
    for s, k in zip(replayed, kept):
        for a, b in zip(s, k):
            a.copy_(b)
    for i in range(5):
        token.fill_(7 * i)
        want, _ = model.run(token, eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(logits, want), i
    assert all(torch.equal(a, b) for s, e in zip(replayed, eager) for a, b in zip(s, e))


def test_another_device_is_current(monkeypatch):
    say("[ssm] another device is current")
    u, w, t = torch.randn(2, 5, 8, device="cuda"), torch.randn(8, 4, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    a, b, h = -torch.rand(8, 4, device="cuda"), torch.randn(2, 5, 1, 4, device="cuda"), torch.zeros(2, 8, 4, device="cuda")
    st, e = torch.zeros(2, 3, 8, device="cuda"), torch.randn(3, 8, device="cuda")
    saved = ssm.ssm_scan_fwd(u, u, a, b, b)[2]
    calls = [lambda: ssm.ssm_scan_fwd(u, u, a, b, b), lambda: ssm.ssm_scan_bwd(u, u, a, b, b, None, None, None, saved, u),
             lambda: ssm.ssm_scan_step(h, u[:, 0], u[:, 0], a, b[:, 0], b[:, 0]), lambda: ssm.causal_conv_fwd(u, w), lambda: ssm.causal_conv_bwd(u, w, None, u),
             lambda: ssm.causal_conv_step(u[:, 0], w, None, st), lambda: lm.embed_fwd(t, e), lambda: lm.embed_bwd(t, e, 9)]
    for f in calls:
        f()
    torch.cuda.synchronize()
    bind = lm._native()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    bind.setup(lambda: 1, torch._C._cuda_getCurrentRawStream)
    try:
        for f in calls:
            with pytest.raises(ValueError, match="the current device is cuda:1"):
                f()
    finally:
        bind.setup(torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    monkeypatch.undo()
    for f in calls:
        f()
    torch.cuda.synchronize()
