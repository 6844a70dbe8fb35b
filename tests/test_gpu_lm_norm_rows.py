"""Block norms, bounded row by row: narrow rows.

FP32 rounds each product and sum by 2^-24 of itself.  r = x + u with u's dozen operations is off by 1e-6 (|x| + |u|), so rh = r rs2 by
1e-6 k (1 + |rh|), k = the row's largest (|x| + |u|) rs2 or 1; everything behind rh carries that, times the terms it is made of.
1e-5 of those terms leaves room for sums of some hundred columns."""
import pytest
import torch

from tests.helpers import say
from tests.test_gpu_lm_norm import EPS, both, make, plain

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def bounds(a, act):
    """The terms of every output, in 64 bits: of a row's outputs the row's own, of a column sum the column's."""
    t = {k: None if v is None else v.cpu().double() for k, v in a.items()}
    y, one = t["y"], torch.ones((), dtype=torch.float64)
    full = t["w_post"] is not None
    w1, sc = (t["w_post"], t["scale"]) if full else (one, one)
    rs1 = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) if full else one
    s = one if t["gate"] is None else torch.sigmoid(t["gate"])
    f, df = (s, one * 0) if t["gate"] is None else (s * t["gate"], s * (1 + t["gate"] * (1 - s))) if act == "silu" else (s, s * (1 - s))
    yh = (y * rs1).abs()
    w1, sc, f, df = w1.abs(), sc.abs(), f.abs(), df.abs()
    u = sc * f * yh * w1
    size = t["x"].abs() + u
    r = plain(dict(a, dr=None, dn=None), act)[0]
    rs2 = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    k = (size * rs2).amax(-1, keepdim=True).clamp_min(1.0)
    rh, p = (r * rs2).abs(), (t["dn"] * t["w_pre"]).abs()
    v = ((t["dr"].abs() + rs2 * (p + rh * (p * rh).mean(-1, keepdim=True))) * k).amax(-1, keepdim=True)
    q = v * sc * f * w1 + 0 * y
    out = dict(r=size, n=k * (1 + rh) * t["w_pre"].abs(), dx=v + 0 * y, dy=rs1 * (q + yh * (q * yh).mean(-1, keepdim=True)) if full else q,
               dw_pre=(t["dn"].abs() * (1 + rh) * k).sum(0))
    if t["gate"] is not None:
        out["dgate"] = v * sc * yh * w1 * (1 + df)
    if full:
        out.update(dw_post=(v * f * yh * sc).sum(0), dscale=(v * f * yh * w1).sum(0))
    return out


def within(got, ref, size, what):
    tol = 1e-5 * size + 2.0 ** -126 + (2.0 ** -8 * ref.abs() if got.dtype == bf else 0.0)
    bad = (got.cpu().double() - ref).abs() - tol
    at = int(bad.reshape(-1).argmax())
    assert float(bad.max()) <= 0, (what, at, float(got.reshape(-1)[at]), float(ref.reshape(-1)[at]), float(size.expand_as(ref).reshape(-1)[at]))


@pytest.mark.parametrize("d", [1, 2, 3, 4, 5, 15, 63, 64, 65, 67, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("rows", [1, 17, 600, 9000])
def test_narrow_rows_by_row(rows, d):
    say(f"[norm] narrow rows by row {rows}x{d}")
    act = ("silu", "sigmoid", "none")[(rows + d) % 3]
    st, br = (bf, f32) if d % 2 else (f32, bf)
    a = make(rows, d, st, br, act, d % 3 != 0, rows + d)
    (r, n, grads), (rr, rn, rg), size = both(a, act), plain(a, act), bounds(a, act)
    within(r, rr, size["r"], "r")
    within(n, rn, size["n"], "n")
    assert set(grads) == set(rg)
    for k in rg:
        within(grads[k], rg[k], size[k], k)
