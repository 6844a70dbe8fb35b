"""Linear cross entropy with logits far beyond the cap, against the definition in 64 bits.

There 1 - tanh^2 is small, and it is the factor of every gradient.  Tolerances: a logit's FP32 sum is off by at most
e_z = 2e-6 of its sum of magnitudes; over the cap that moves 1 - tanh^2 by 2 e_z / cap of itself, and each of lse and the
capped logit by no more than e_z and 4e-7 of the cap, so the probability by twice that.  exp2 of an argument up to 36 is off by 36 2^-24
and a few roundings: 1e-5.  dz is rounded to BF16, 2^-8 of the term; BF16 gradients are rounded once more."""
import pytest
import torch

from linear_recurrence_sequence_amd import lm
from tests.helpers import say
from tests.test_gpu_lm_ce import within

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("n", [20, 200, 700])
@pytest.mark.parametrize("grad_dtype", [f32, bf], ids=["f32", "bf16"])
@pytest.mark.parametrize("zloss", [False, True])
@pytest.mark.parametrize("low,high", [(0.5, 3.0), (6.0, 12.0)])
def test_saturated_logits(n, grad_dtype, zloss, low, high):
    """Every logit between low and high times the cap, of either sign."""
    say(f"[ce] logits {low} to {high} caps, n={n} {grad_dtype} zloss={zloss}")
    cap, d, v = 2.0, 64, 900
    g = torch.Generator(device="cuda").manual_seed(n)

    def u(*shape, lo=0.0, hi=1.0):
        return lo + (hi - lo) * torch.rand(*shape, generator=g, device="cuda")

    sign = torch.where(u(v) < 0.5, -1.0, 1.0)
    root = (high / low) ** 0.25                       # z / cap = a b over low..high
    a, b = u(n, lo=low * root, hi=high / root), u(v, lo=1.0 / root, hi=root) * sign
    h = (cap * a[:, None] * u(n, d, lo=0.98, hi=1.02)).to(bf)
    w = (b[:, None] * u(v, d, lo=0.98, hi=1.02) / d).to(bf)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[::5] = -1
    dloss, dlse = u(n, lo=0.5) / n, 1e-1 * u(n, lo=-0.5, hi=0.5) / n
    h64, w64, row = h.double(), w.double(), torch.arange(n, device="cuda")
    z = h64 @ w64.t()
    assert float(z.abs().min()) > 0.8 * low * cap and float(z.abs().max()) < 1.2 * high * cap
    ez = 2e-6 * (h64.abs() @ w64.abs().t()).max()
    th = torch.tanh(z / cap)
    slope, z = 1.0 / torch.cosh(z / cap) ** 2, cap * th
    lse = torch.logsumexp(z, 1)
    dl = torch.where(t >= 0, dloss.double(), torch.zeros_like(lse))
    c = dl + dlse.double() if zloss else dl
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros_like(p)
    hot[row, t.clamp_min(0)] = 1.0
    dz, mag = (p * c[:, None] - hot * dl[:, None]) * slope, (p * c.abs()[:, None] + hot * dl[:, None]) * slope
    rel = 2.0 ** -8 + float(2 * ez / cap + 2 * (ez + 4e-7 * cap)) + 1e-5
    _, e = lm.linear_ce_fwd(h, w, t, softcap=cap)
    got = lm.linear_ce_bwd(h, w, t, e, dloss, dlse if zloss else None, softcap=cap, grad_dtype=grad_dtype)
    within(got["dh"], dz @ w64, rel * (mag @ w64.abs()), "dh")
    within(got["dw"], dz.t().contiguous() @ h64, rel * (mag.t().contiguous() @ h64.abs()), "dw")


def test_logits_without_an_end():
    """Infinite logits are the cap itself: the gradient through them is zero, and nothing becomes NaN."""
    say("[ce] infinite logits under a cap")
    n, d, v, cap = 40, 16, 300, 5.0
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randn(v, d, generator=g, device="cuda").to(bf)
    h = torch.randn(n, d, generator=g, device="cuda").to(bf)
    w[:, 0] = w[:, 0].abs() + 1
    h[::2, 0] = 3e38                                    # FP32 sums beyond its range
    w[:, 0] *= 100
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    loss, lse = lm.linear_ce_fwd(h, w, t, softcap=cap)
    got = lm.linear_ce_bwd(h, w, t, lse, torch.ones(n, device="cuda"), softcap=cap, grad_dtype=f32)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(got["dh"]).all())
    assert bool((got["dh"][::2] == 0).all()) and bool((got["dh"][1::2] != 0).any())
