"""The 64-bit definitions that the GPU tests go by, against automatic differentiation and against differences (CPU)."""
import pytest
import torch

from tests.ssm_ref import conv_ref, scan_ref

f64 = torch.float64


def scan_inputs(batch=2, length=7, width=6, n=3, groups=2, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=f64)

    k = dict(u=normal(batch, length, width), dt=normal(batch, length, width), a=-normal(width, n).abs() - 0.1, b=normal(batch, length, groups, n),
             c=normal(batch, length, groups, n), d=normal(width), z=normal(batch, length, width), dt_bias=normal(width),
             h0=normal(batch, width, n))
    return k, normal(batch, length, width), normal(batch, width, n)


@pytest.mark.parametrize("plain", [False, True])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients(plain, softplus):
    k, dy, dh = scan_inputs()
    kw = dict(softplus=softplus)
    if not plain:
        kw["reset"] = torch.tensor([[0, 0, 1, 0, 1, 1, 0], [1, 0, 0, 0, 0, 0, 1]], dtype=torch.uint8)
        kw["lengths"] = torch.tensor([7, 5], dtype=torch.int32)
    want = scan_ref(**k, **kw, dy=dy, dh_final=dh)
    leaf = {n: t.clone().requires_grad_() for n, t in k.items()}

    def loss(**x):
        r = scan_ref(**x, **kw)
        return (r["y"] * dy).sum() + (r["h"] * dh).sum()

    got = torch.autograd.grad(loss(**leaf), list(leaf.values()))
    names = dict(a="da", u="du", dt="ddt", b="db", c="dc", d="dd", z="dz", dt_bias="ddt_bias", h0="dh0")
    for n, t in zip(leaf, got):
        torch.testing.assert_close(want[names[n]], t, rtol=1e-12, atol=1e-12)
    g = torch.Generator().manual_seed(1)
    # The losses' own roundings: 120 terms are added up, each with fewer than 80 roundings of 2^-53 behind it, so that a loss is off by
    # less than 200 * 2^-53 of the sum of its terms' sizes (large where softplus is off: steps of either sign make states grow).
    sized = scan_ref(**k, **kw, absolute=True)
    rounding = 200 * 2.0 ** -53 * float((sized["y"] * dy.abs()).sum() + (sized["h"] * dh.abs()).sum())
    for n in k:                                   # a step of 2^-17 leaves 2^-34 times third derivatives
        step = torch.randn(k[n].shape, generator=g, dtype=f64) * 2.0 ** -17
        diff = float(loss(**{**k, n: k[n] + step}) - loss(**{**k, n: k[n] - step})) / 2
        along = float((want[names[n]] * step).sum())
        assert abs(diff - along) < 1e-8 * (1 + abs(along)) + rounding


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("length", [1, 2, 6])
def test_conv_gradients(silu, width, length):
    g = torch.Generator().manual_seed(length)

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=f64)

    k = dict(x=normal(2, length, 5), w=normal(5, width), bias=normal(5), state=normal(2, width - 1, 5))
    dy, do = normal(2, length, 5), normal(2, width - 1, 5)
    kw = dict(silu=silu, reset=(torch.rand(2, length, generator=g) < 0.3).to(torch.uint8), lengths=torch.tensor([length, length // 2], dtype=torch.int32))
    want = conv_ref(**k, **kw, dy=dy, dstate_out=do)
    leaf = {n: t.clone().requires_grad_() for n, t in k.items()}
    r = conv_ref(**leaf, **kw)
    got = torch.autograd.grad((r["y"] * dy).sum() + (r["last"] * do).sum(), list(leaf.values()))
    for n, t in zip(("dx", "dw", "dbias", "dstate"), got):
        torch.testing.assert_close(want[n], t, rtol=1e-12, atol=1e-12)


def test_a_row_in_two_parts():
    """A scan that goes on from a state, and a convolution that does, are those of the whole row."""
    k, _, _ = scan_inputs()
    whole = scan_ref(**k)
    rows = ("u", "dt", "b", "c", "z")
    first = scan_ref(**{n: t[:, :4] if n in rows else t for n, t in k.items()})
    rest = scan_ref(**{**{n: t[:, 4:] if n in rows else t for n, t in k.items()}, "h0": first["h"]})
    torch.testing.assert_close(torch.cat([first["y"], rest["y"]], 1), whole["y"], rtol=1e-12, atol=1e-12)
    x, w = torch.randn(2, 9, 3, dtype=f64), torch.randn(3, 4, dtype=f64)
    one = conv_ref(x, w)
    a = conv_ref(x[:, :2], w)
    b = conv_ref(x[:, 2:], w, state=a["last"])
    torch.testing.assert_close(torch.cat([a["y"], b["y"]], 1), one["y"], rtol=1e-12, atol=1e-12)
