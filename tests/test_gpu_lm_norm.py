"""Block norms on the GPU against the definition in 64 bits.

Tolerances: arithmetic is FP32 with sums over d terms, so an FP32 output is
within a few dozen units of 2^-24 of its scale; 1e-5 of the largest value of
the reference is a bound with room.  A BF16 output adds one rounding, at most
2^-8 of the value, element by element.  Column sums over n rows of FP32 products: 1e-5
of the sum of magnitudes.  Below FP32's least normal value, 2^-126, the format
itself holds nothing to 1e-5: that much is allowed on every element."""
import pytest
import torch

from linear_recurrence_sequence_amd import autograd, lm
from tests.helpers import say

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32
EPS = 1e-6


def make(rows, d, st, br, gate, full, seed):
    g = torch.Generator().manual_seed(seed)

    def n(shape, dt, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g) * std + mean).to(dt).cuda()

    return dict(x=n((rows, d), st, 2.0), y=n((rows, d), br, 1.5), gate=None if gate == "none" else n((rows, d), br),
                w_post=n(d, f32, 0.1, 1.0) if full else None, scale=n(d, f32, 0.1, 0.5) if full else None,
                w_pre=n(d, f32, 0.1, 1.0), dr=n((rows, d), st), dn=n((rows, d), br))


def plain(a, act, eps=EPS):
    """The definition in 64 bits on the CPU, differentiated by autograd."""
    names = [k for k in ("x", "y", "gate", "w_post", "scale", "w_pre") if a[k] is not None]
    t = {k: a[k].detach().cpu().double().requires_grad_() for k in names}

    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w

    u = norm(t["y"], t["w_post"]) if "w_post" in t else t["y"]
    if "gate" in t:
        s = torch.sigmoid(t["gate"])
        u = u * (s * t["gate"] if act == "silu" else s)
    if "scale" in t:
        u = u * t["scale"]
    r = t["x"] + u
    n = norm(r, t["w_pre"])
    cot = [torch.zeros_like(r) if a[k] is None else a[k].cpu().double() for k in ("dr", "dn")]
    grads = torch.autograd.grad([r, n], [t[k] for k in names], cot)
    return r.detach(), n.detach(), {"d" + k: g for k, g in zip(names, grads)}


def close(got, ref, what, scale=None):
    got, ref_t = got.detach().cpu().double(), ref
    assert got.shape == ref_t.shape, what
    if not got.numel():
        return
    top = float(ref_t.abs().max()) if scale is None else scale
    tol = 1e-5 * top + 2.0 ** -126 + (2.0 ** -8 * ref_t.abs() if what.endswith("bf16") else 0.0)
    bad = (got - ref_t).abs() - tol
    assert float(bad.max()) <= 0, (what, float((got - ref_t).abs().max()), top)


def tag(t, name):
    return name + (" bf16" if t.dtype == bf else " f32")


def check(a, act, got, ref):
    r, n, grads = got
    rr, rn, rg = ref
    close(r, rr, tag(r, "r"))
    close(n, rn, tag(n, "n"))
    rows = max(1, a["x"].shape[0])
    for k in rg:
        # a column sum's FP32 partials are off relative to the size of its terms, not of the sum
        scale = max(float(rg[k].abs().max()), 4.0 * rows ** 0.5) if k in ("dw_post", "dscale", "dw_pre") else None
        close(grads[k], rg[k], tag(grads[k], k), scale)
    assert set(grads) == set(rg)


def both(a, act, **kw):
    w = [a[k] for k in ("x", "y", "gate", "w_post", "scale", "w_pre")]
    r, n, stats = lm.block_norm_fwd(*w, eps=EPS, gate_act=act, **kw)
    return r, n, lm.block_norm_bwd(*w, stats, a["dr"], a["dn"], eps=EPS, gate_act=act)


@pytest.mark.parametrize("st,br", [(bf, bf), (f32, bf), (f32, f32), (bf, f32)], ids=["bb", "fb", "ff", "bf"])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 3), (3, 8), (5, 63), (2, 64), (9, 255), (4, 256), (7, 257), (600, 260), (513, 511),
                                    (515, 1000), (33, 1537), (17, 2048), (520, 2560), (6, 4096), (5, 4099), (3, 8192),
                                    (2, 8195), (3, 16384)])
def test_shapes(rows, d, st, br):
    say(f"[norm] rows={rows} d={d} {st} {br}")
    # every form is met over the shapes
    act = ("silu", "sigmoid", "none")[(rows + d) % 3]
    full = (rows * d) % 2 == 0
    a = make(rows, d, st, br, act, full, rows * 100003 + d)
    check(a, act, both(a, act), plain(a, act))


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("full", [True, False], ids=["full", "plain"])
def test_forms(act, full):
    for rows, d in ((1500, 320), (1030, 96), (40, 320)):
        say(f"[norm] {act} full={full} {rows}x{d}")
        a = make(rows, d, f32, bf, act, full, 5)
        check(a, act, both(a, act), plain(a, act))


def test_rows_of_a_wider_projection():
    """y and gate are halves of one projection, x and the cotangents strided rows."""
    say("[norm] strided rows")
    rows, d = 77, 136
    a = make(rows, d, bf, bf, "silu", True, 9)
    wide = torch.cat([a["y"], a["gate"]], 1)
    b = dict(a, y=wide[:, :d], gate=wide[:, d:])
    for k in ("x", "dr", "dn"):
        b[k] = torch.cat([a[k], a[k][:, :3]], 1)[:, :d]       # odd row stride: rows start off any 16-byte line
        assert b[k].stride(0) == d + 3
    want, got = both(a, "silu"), both(b, "silu")
    for u, w in zip(got[:2], want[:2]):
        assert torch.equal(u, w)
    for k in want[2]:
        assert torch.equal(got[2][k], want[2][k]), k
    # [B, L, d] with both leading strides of the wide rows
    w3 = wide.view(7, 11, 2 * d)
    args = (a["x"].view(7, 11, d), w3[..., :d], w3[..., d:], a["w_post"], a["scale"], a["w_pre"])
    r3, n3, _ = lm.block_norm_fwd(*args, eps=EPS, gate_act="silu")
    assert r3.shape == (7, 11, d) and torch.equal(r3.view(rows, d), want[0]) and torch.equal(n3.view(rows, d), want[1])


def test_broadcast_gate_row_and_in_place_stream():
    say("[norm] one gate row for all, r into x")
    rows, d = 21, 200
    a = make(rows, d, f32, bf, "sigmoid", True, 10)
    a["gate"] = a["gate"][:1].expand(rows, d)
    ref = plain(a, "sigmoid")
    x = a["x"].clone()
    r, n, _ = lm.block_norm_fwd(x, a["y"], a["gate"], a["w_post"], a["scale"], a["w_pre"], eps=EPS,
                                gate_act="sigmoid", r=x)
    assert r.data_ptr() == x.data_ptr()
    close(r, ref[0], "r f32")
    close(n, ref[1], "n bf16")
    # the gradient of the broadcast row is the sum over the rows
    leaf = a["gate"][:1].detach().clone().requires_grad_()
    r, n = autograd.block_norm(a["x"], a["y"], leaf.expand(rows, d), a["w_post"], a["scale"], a["w_pre"], eps=EPS,
                               gate_act="sigmoid")
    torch.autograd.backward([r, n], [a["dr"], a["dn"]])
    want = ref[2]["dgate"].sum(0, keepdim=True)
    # 21 BF16-rounded terms and torch's BF16 result
    tol = 2.0 ** -8 * (ref[2]["dgate"].abs().sum(0, keepdim=True) + want.abs()) + 1e-4
    assert bool(((leaf.grad.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("rows", [0, 1])
def test_missing_cotangents_and_no_rows(rows):
    say(f"[norm] rows={rows}, cotangents missing")
    a = make(rows, 40, f32, f32, "silu", True, 11)
    for k in ("dr", "dn"):
        b = dict(a, **{k: None})
        check(b, "silu", both(b, "silu"), plain(b, "silu"))


def test_zero_rows_and_extremes():
    """An all-zero branch, gates at both ends of sigmoid, values whose squares are near FP32's ends."""
    say("[norm] zeros and extremes")
    d = 72
    a = make(6, d, f32, f32, "silu", True, 12)
    a["y"][0] = 0.0
    a["gate"][1] = 100.0
    a["gate"][2] = -100.0
    a["y"][3] *= 1e15
    a["y"][4] *= 1e-15
    a["x"][5] = 0.0
    a["y"][5] = 0.0
    r, n, g = both(a, "silu")
    rr, rn, rg = plain(a, "silu")
    for k in range(6):          # row by row, each on its own scale
        close(r[k], rr[k], "r f32")
        close(n[k], rn[k], "n f32")
        for name in ("dx", "dy", "dgate"):
            close(g[name][k], rg[name][k], name + " f32")
    assert all(bool(torch.isfinite(t).all()) for t in (r, n, *g.values()))


def test_differences():
    """The gradient against central differences of the forward, FP32."""
    say("[norm] differences")
    a = make(3, 24, f32, f32, "silu", True, 13)
    _, _, g = both(a, "silu")
    gen = torch.Generator().manual_seed(1)

    def value(b):
        r, n, _ = lm.block_norm_fwd(b["x"], b["y"], b["gate"], b["w_post"], b["scale"], b["w_pre"], eps=EPS, gate_act="silu")
        return float((r.double() * a["dr"].double()).sum() + (n.double() * a["dn"].double()).sum())

    h = 1e-2
    for k in ("x", "y", "gate", "w_post", "scale", "w_pre"):
        e = torch.randn(a[k].shape, generator=gen).cuda()
        got = (value(dict(a, **{k: a[k] + h * e})) - value(dict(a, **{k: a[k] - h * e}))) / (2 * h)
        want = float((g["d" + k].double() * e.double()).sum())
        # h^2 of third derivatives (a few units of the sum of ~72 terms) and 1e-6 / h of FP32 rounding
        assert abs(got - want) <= 2e-2 * max(1.0, float((g["d" + k] * e).abs().sum())), (k, got, want)


def test_autograd_stream_and_graph():
    """Through autograd, on a side stream, and replayed from a graph with eager work between the replays."""
    say("[norm] autograd, side stream, graph")
    a = make(300, 192, bf, bf, "silu", True, 14)
    want = both(a, "silu")
    leaves = {k: a[k].clone().requires_grad_() for k in ("x", "y", "gate", "w_post", "scale", "w_pre")}
    r, n = autograd.block_norm(*leaves.values(), eps=EPS, gate_act="silu")
    torch.autograd.backward([r, n], [a["dr"], a["dn"]])
    assert torch.equal(r, want[0]) and torch.equal(n, want[1])
    for k, t in leaves.items():
        assert torch.equal(t.grad, want[2]["d" + k]), k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(a, "silu")
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2]["dw_pre"], want[2]["dw_pre"])
    with torch.cuda.stream(side):
        both(a, "silu")
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = both(a, "silu")
    for rep in range(3):
        for t in (out[0], out[1], *out[2].values()):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), rep
        for k in want[2]:
            assert torch.equal(out[2][k], want[2][k]), (rep, k)
        both(a, "silu")


@pytest.mark.parametrize("rows,d", [(513, 513), (1030, 770), (600, 1023), (2500, 1024), (700, 1021), (1200, 1025), (300, 6145)])
@pytest.mark.parametrize("st,br", [(bf, bf), (f32, f32)], ids=["bb", "ff"])
def test_a_wave_a_row(rows, d, st, br):
    """Widths around the border between one wave and several a row, with rows to spare and without."""
    say(f"[norm] wave a row {rows}x{d} {st}")
    act = ("silu", "sigmoid", "none")[rows % 3]
    a = make(rows, d, st, br, act, d % 2 == 0, rows + d)
    check(a, act, both(a, act), plain(a, act))


def term_sizes(a, act, eps=EPS):
    """What FP32's roundings are to be measured by over few columns, where results cancel, in 64 bits.  r = x + u may be
    far smaller than x and u, and norm(r) divides by it: everything behind it carries r's rounding k = (|x| + |u|) rs2 times.
    A norm's gradient is a difference that over one column cancels but for eps's part.  So: the largest of the terms of
    n, dx, dy and dgate, times k, and the sums of the magnitudes of the weights' gradients, times k."""
    t = {k: None if v is None else v.cpu().double() for k, v in a.items()}
    y, one = t["y"], torch.ones((), dtype=torch.float64)
    w1, sc = (one, one) if t["w_post"] is None else (t["w_post"], t["scale"])
    rs1 = one if t["w_post"] is None else 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    g = torch.sigmoid(t["gate"]) if t["gate"] is not None else one
    f, df = (g, one * 0) if t["gate"] is None else (g * t["gate"], g * (1 + t["gate"] * (1 - g))) if act == "silu" else (g, g * (1 - g))
    yh = y * rs1
    u = sc * f * yh * w1
    r = t["x"] + u
    rs2 = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    k = ((t["x"].abs() + u.abs()) * rs2).amax(-1, keepdim=True).clamp_min(1.0)
    p = (t["dn"] * t["w_pre"]).abs()
    rh = (r * rs2).abs()
    v = (t["dr"].abs() + rs2 * (p + rh * (p * rh).mean(-1, keepdim=True))) * k
    q = v * (sc * f * w1).abs()
    dy = q if t["w_post"] is None else rs1 * (q + yh.abs() * (q * yh.abs()).mean(-1, keepdim=True))
    out = dict(n=k * (t["w_pre"].abs() + 0 * rh), dx=v, dy=dy, dgate=v * (sc * yh * w1 * df).abs())
    out = {key: float(x.max()) for key, x in out.items()}
    out["dw_pre"] = float((t["dn"].abs() * rh * k).sum(0).max())
    s = (v * (f * yh).abs()).sum(0)
    out.update(dw_post=float((s * sc).abs().max()), dscale=float((s * w1).abs().max()))
    return out


@pytest.mark.parametrize("d", [1, 2, 3, 4, 5, 15, 63, 64, 65, 67, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("rows", [1, 17, 600, 9000])
def test_narrow_rows(rows, d):
    """Several rows to a wave, and every remainder of the width by four."""
    say(f"[norm] narrow rows {rows}x{d}")
    act = ("silu", "sigmoid", "none")[(rows + d) % 3]
    st, br = (bf, f32) if d % 2 else (f32, bf)
    a = make(rows, d, st, br, act, d % 3 != 0, rows + d)
    (r, n, grads), (rr, rn, rg), size = both(a, act), plain(a, act), term_sizes(a, act)
    close(r, rr, tag(r, "r"))
    close(n, rn, tag(n, "n"), size["n"])
    assert set(grads) == set(rg)
    for k in rg:
        close(grads[k], rg[k], tag(grads[k], k), size[k])
