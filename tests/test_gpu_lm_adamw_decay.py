"""The decay of AdamW where lr * decay is small against one, and of weights that are not finite.

Tolerance: the new weight is rounded to FP32 once, half a unit in its last place; what is taken from it is far smaller and
off by a few roundings of itself, 2e-6 of the decay and of the step."""
import math

import pytest
import torch

from linear_recurrence_sequence_amd import lm
from tests.helpers import say

pytestmark = pytest.mark.gpu
LR = 1e-3


def half_unit(x):
    return torch.ldexp(torch.ones_like(x), torch.frexp(x).exponent - 25)


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("moving", [False, True])
@pytest.mark.parametrize("taken", [1e-3, 1e-5, 1e-6, 1e-7, 5e-8, 3e-8, 2e-8])
def test_small_decays(taken, moving, master):
    say(f"[adamw] lr decay = {taken}, moving={moving} master={master}")
    n = 10000
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(n, generator=g)).cuda()
    grad = (1e-3 * torch.randn(n, generator=g)).cuda() if moving else torch.zeros(n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    w64, g64 = w.cpu().double(), grad.cpu().double()
    lr, b1, b2 = (LR, 0.9, 0.95) if not moving else (1e-7, 0.9, 0.95)
    step = lr * g64 / (g64.abs() + 1e-8)                # the first step, from zero moments
    want = w64 - taken * w64 - step
    kept = w.clone() if master else None
    p = w.bfloat16() if master else w
    lm.adamw_step([p], [grad], [m], [v], step=1, lr=lr, betas=(b1, b2), eps=1e-8, weight_decay=taken / lr,
                  masters=[kept] if master else None)
    got = (kept if master else p).cpu().double()
    bad = (got - want).abs() - half_unit(torch.maximum(want.abs(), w64.abs())) - 2e-6 * (taken * w64.abs() + step.abs())
    assert float(bad.max()) <= 0, float(bad.max() / half_unit(want.abs()).max())
    if master:
        assert torch.equal(p, kept.bfloat16())


@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_weights_that_are_not_finite(decay):
    """p (1 - lr decay) of an infinite weight is infinite, of NaN NaN; the neighbours take their step."""
    say(f"[adamw] infinite weights, decay={decay}")
    p = torch.ones(600, device="cuda")
    p[3], p[300], p[599], p[7] = math.inf, -math.inf, math.nan, 3.4e38
    g = torch.full((600,), 1e-3, device="cuda")
    lm.adamw_step([p], [g], [torch.zeros(600, device="cuda")], [torch.zeros(600, device="cuda")], step=1, lr=LR, betas=(0.9, 0.95),
                  weight_decay=decay)
    p = p.cpu()
    assert p[3] == math.inf and p[300] == -math.inf and math.isnan(p[599])
    assert torch.isfinite(p).sum() == 597 and abs(float(p[7]) / 3.4e38 - (1 - LR * decay)) < 2e-7
    assert abs(float(p[0]) - (1 - LR * decay - LR)) < 2e-7
