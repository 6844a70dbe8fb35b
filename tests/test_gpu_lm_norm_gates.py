"""Block norms with gates far from zero, element by element."""
import pytest
import torch

from tests.helpers import say
from tests.test_gpu_lm_norm import both, make

pytestmark = pytest.mark.gpu
f32 = torch.float32


@pytest.mark.parametrize("rows,d", [(6, 40), (700, 260), (5, 2050)])
def test_gates_far_from_zero(rows, d):
    """sigmoid' = s (1 - s) of a large gate is small, and all that dgate is.  Without a norm on the branch, and from dr alone,
    dgate = dr y s (1 - s).  exp2 takes 1.44 |g| <= 26, off by 2^-24 of itself twice (3.2e-6 of the result at most, over ln 2), and a
    dozen roundings stand around it: 4e-6."""
    say(f"[norm] large gates {rows}x{d}")
    a = make(rows, d, f32, f32, "sigmoid", False, rows)
    g = torch.Generator().manual_seed(2)
    a["gate"] = ((16.0 * torch.rand(rows, d, generator=g) + 2.0) * torch.where(torch.rand(rows, d, generator=g) < 0.5, -1.0, 1.0)).cuda()
    a["dn"] = None
    got = both(a, "sigmoid")[2]["dgate"].cpu().double()
    e = torch.exp(-a["gate"].cpu().double().abs())
    want = (a["dr"].double() * a["y"].double()).cpu() * e / (1 + e) ** 2
    assert bool(((got - want).abs() <= 4e-6 * want.abs()).all())
    a["gate"][0, :4] = torch.tensor([200.0, -200.0, float("inf"), -float("inf")])
    assert bool((both(a, "sigmoid")[2]["dgate"][0, :4] == 0).all())
