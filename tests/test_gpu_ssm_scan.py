"""The selective scan on the GPU against its definition in 64 bits: forward, backward and single tokens."""
import pytest
import torch

from linear_recurrence_sequence_amd import autograd, ssm
from tests.helpers import say
from tests.ssm_ref import scan_ref, scan_tolerance

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32
ROWS = ("u", "dt", "b", "c", "z")


def inputs(batch, length, width, n, groups, dtype, seed=0, gate=True, full=True, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dt=f32, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    k = dict(u=normal(batch, length, width, dt=dtype), dt=normal(batch, length, width, dt=dtype, std=scale),
             a=-torch.rand(width, n, generator=g, device="cuda") * 4 - 0.05, b=normal(batch, length, groups, n, dt=dtype),
             c=normal(batch, length, groups, n, dt=dtype), d=normal(width) if full else None,
             z=normal(batch, length, width, dt=dtype) if gate else None, dt_bias=normal(width) - 2 if full else None,
             h0=normal(batch, width, n) if full else None)
    return k, normal(batch, length, width, dt=dtype), normal(batch, width, n) if full else None


def flags(batch, length, seed, p=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(batch, length, generator=g, device="cuda") < p).to(torch.uint8)


def run(k, dy, dh, **kw):
    args = [k[n] for n in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")]
    y, h, saved = ssm.ssm_scan_fwd(*args, k["h0"], **kw)
    out = dict(y=y, h=h)
    if dy is not None:
        out.update(ssm.ssm_scan_bwd(*args, saved, dy, dh, want_dh0=k["h0"] is not None, **kw))
    torch.cuda.synchronize()
    return out


def check(got, k, dy, dh, kw, dtype, length):
    ref = scan_ref(**k, **kw, dy=dy, dh_final=dh)
    tol = scan_tolerance(scan_ref(**k, **kw, dy=dy, dh_final=dh, absolute=True), ref, length, dtype)
    for n, t in got.items():
        assert t.shape == ref[n].shape and t.dtype == (f32 if n in ("h", "da", "dd", "ddt_bias", "dh0") else dtype)
        err = (t.double() - ref[n]).abs()
        bad = ~(err <= tol[n])
        assert not bad.any(), (n, int(bad.sum()), float(err.max()), float((err / tol[n]).max()))


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,length,width,n,groups", [
    (1, 1, 1, 1, 1), (2, 1, 70, 16, 1), (1, 15, 33, 16, 1), (1, 16, 32, 16, 1), (3, 17, 34, 16, 2), (2, 70, 64, 4, 1), (2, 33, 130, 3, 1),
    (2, 37, 129, 8, 3), (1, 50, 96, 5, 2), (2, 41, 40, 32, 1), (1, 35, 17, 17, 1), (2, 23, 24, 64, 2), (1, 40, 9, 33, 1), (1, 300, 48, 16, 1),
    (5, 64, 12, 13, 4), (1, 19, 515, 16, 1),
])
def test_parity(dtype, batch, length, width, n, groups):
    say(f"[ssm] {dtype} batch={batch} length={length} width={width} n={n} groups={groups}")
    k, dy, dh = inputs(batch, length, width, n, groups, dtype, seed=length)
    check(run(k, dy, dh), k, dy, dh, {}, dtype, length)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate,full,softplus", [(False, True, True), (True, False, True), (False, False, True), (True, True, False)])
def test_forms(dtype, gate, full, softplus):
    say(f"[ssm] forms {dtype} gate={gate} full={full} softplus={softplus}")
    k, dy, dh = inputs(2, 39, 50, 16, 1, dtype, seed=3, gate=gate, full=full)
    if not softplus:
        k["dt"] = k["dt"].abs() * 0.3
        if full:
            k["dt_bias"] = k["dt_bias"].abs() * 0.1
    kw = dict(softplus=softplus)
    check(run(k, dy, dh, **kw), k, dy, dh, kw, dtype, 39)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,length,width,n", [(2, 45, 36, 16), (1, 200, 20, 16), (3, 16, 20, 4), (2, 33, 20, 40)])
def test_packed_and_padded(dtype, batch, length, width, n):
    say(f"[ssm] packed and padded {dtype} batch={batch} length={length} width={width} n={n}")
    k, dy, dh = inputs(batch, length, width, n, 1, dtype, seed=5)
    lengths = torch.tensor([length // 2, length, 0][:batch], dtype=torch.int32, device="cuda")
    for kw in (dict(reset=flags(batch, length, 1)), dict(lengths=lengths), dict(reset=flags(batch, length, 2).bool(), lengths=lengths),
               dict(reset=torch.ones(batch, length, dtype=torch.uint8, device="cuda")),
               dict(lengths=torch.tensor([-3, length + 9, 1][:batch], dtype=torch.int32, device="cuda"))):
        check(run(k, dy, dh, **kw), k, dy, dh, kw, dtype, length)


def test_nothing_crosses_a_start_or_comes_from_padding():
    """What stands before a sequence's start, and in padding, may be NaN or infinite."""
    say("[ssm] NaN before a start and in padding")
    k, dy, dh = inputs(2, 60, 40, 16, 1, bf, seed=8)
    reset = torch.zeros(2, 60, dtype=torch.uint8, device="cuda")
    reset[:, 25] = 1
    lengths = torch.tensor([50, 41], dtype=torch.int32, device="cuda")
    kw = dict(reset=reset, lengths=lengths)
    want = run(k, dy, dh, **kw)
    for bad in (float("nan"), float("inf")):
        p = {n: t.clone() for n, t in k.items()}
        py = dy.clone()
        for n in ROWS:
            for i, end in enumerate((50, 41)):
                p[n][i, end:] = bad
        for i, end in enumerate((50, 41)):
            py[i, end:] = bad
        got = run(p, py, dh, **kw)
        for n in want:
            assert torch.equal(got[n], want[n]), n
        for n in ("u", "b", "c", "z"):
            p[n][:, 7] = bad
        p["h0"][:] = bad
        got = run(p, py, dh, **kw)
        for n in ("y", "du", "ddt", "dz", "db", "dc"):
            assert torch.equal(got[n][:, 25:], want[n][:, 25:]), n
        assert torch.equal(got["h"], want["h"])
        late = py.clone()
        late[:, 30] = bad                                      # a cotangent behind the start reaches nothing before it
        got = run(k, torch.where(py.isfinite(), late, dy), dh, **kw)
        for n in ("du", "ddt", "dz", "db", "dc"):
            assert torch.equal(got[n][:, :25], want[n][:, :25]), n
        assert torch.equal(got["dh0"], want["dh0"])


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_steps_of_extreme_size(dtype):
    """A step masked by the type's lowest value or minus infinity leaves the state as it is; a large one forgets all of it, an
    infinite one's token is not finite, and nothing of it is left behind the next start."""
    say(f"[ssm] extreme steps {dtype}")
    k, dy, dh = inputs(2, 40, 30, 16, 1, dtype, seed=70)
    k["dt"][:, 5] = torch.finfo(dtype).min
    k["dt"][:, 11:14] = float("-inf")
    k["dt"][0, 20] = -120.0
    k["dt"][1, 21] = -95.0
    k["dt"][:, 25] = 300.0
    check(run(k, dy, dh), k, dy, dh, {}, dtype, 40)
    state = k["h0"].clone()
    ssm.ssm_scan_step(state, *[k[n] if n in ("a", "d", "dt_bias") else k[n][:, 12] for n in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")])
    assert torch.equal(state, k["h0"])
    k["dt"][:, 30] = float("inf")
    kw = dict(reset=torch.zeros(2, 40, dtype=torch.uint8, device="cuda"))
    kw["reset"][:, 33] = 1
    assert run(k, dy, dh, **kw)["y"][:, 33:].isfinite().all()


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_rows_that_lie_apart(dtype):
    """Parts of wider projections, at offsets of one element, and expanded rows."""
    say(f"[ssm] strides {dtype}")
    batch, length, width, n, groups = 2, 37, 22, 6, 2
    k, dy, dh = inputs(batch, length, width, n, groups, dtype, seed=9)
    want = run(k, dy, dh)
    wide = {}
    for name in ROWS:
        w = k[name].flatten(2).shape[-1]
        buf = torch.full((batch, length, w + 9), float("nan"), dtype=dtype, device="cuda")
        buf[..., 3:3 + w] = k[name].flatten(2)
        wide[name] = buf[..., 3:3 + w].unflatten(-1, k[name].shape[2:])
    buf = torch.full((batch, length, width + 1), float("nan"), dtype=dtype, device="cuda")
    buf[..., 1:] = dy
    got = run({**k, **wide}, buf[..., 1:], dh)
    for name in want:
        assert torch.equal(got[name], want[name]), name
    k["u"] = k["u"][:1, :1].expand(batch, length, width)
    got, want = run(k, dy, dh), run({**k, "u": k["u"].contiguous()}, dy, dh)
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,width,n,groups", [(1, 1, 1, 1), (3, 33, 16, 1), (2, 64, 16, 2), (5, 20, 5, 4), (2, 30, 64, 1), (1, 7, 33, 1), (4, 100, 8, 1)])
def test_step(dtype, batch, width, n, groups):
    say(f"[ssm] step {dtype} batch={batch} width={width} n={n} groups={groups}")
    k, _, _ = inputs(batch, 3, width, n, groups, dtype, seed=11)
    ref = scan_ref(**k)
    tol = scan_tolerance(scan_ref(**k, absolute=True), ref, 3, dtype)
    h = k["h0"].clone()
    for t in range(3):
        y = ssm.ssm_scan_step(h, *[k[m] if k[m] is None or m not in ROWS else k[m][:, t] for m in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")])
        assert y.dtype == dtype and ((y.double() - ref["y"][:, t]).abs() <= tol["y"][:, t]).all()
    assert ((h.double() - ref["h"]).abs() <= tol["h"]).all()
    plain = ssm.ssm_scan_step(h, k["u"][:, 0], k["dt"][:, 0], k["a"], k["b"][:, 0], k["c"][:, 0])
    assert plain.shape == (batch, width) and plain.isfinite().all()


def test_segments_are_the_row():
    """A row long enough to be cut into segments equals the same row walked in parts that are not."""
    say("[ssm] segments")
    k, dy, dh = inputs(1, 2000, 64, 16, 1, f32, seed=12, scale=0.3)
    kw = dict(reset=flags(1, 2000, 4, 0.001))
    got = run(k, dy, dh, **kw)
    check(got, k, dy, dh, kw, f32, 2000)
    h, ys = k["h0"], []
    for t in range(0, 2000, 250):
        part = {n: v[:, t:t + 250] if n in ROWS else v for n, v in k.items()}
        r = run({**part, "h0": h}, None, None, reset=kw["reset"][:, t:t + 250].contiguous())
        h = r["h"]
        ys.append(r["y"])
    torch.testing.assert_close(torch.cat(ys, 1), got["y"], rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(h, got["h"], rtol=1e-4, atol=1e-4)


def test_empty():
    say("[ssm] nothing to do")
    k, dy, dh = inputs(0, 5, 8, 4, 1, f32)
    out = run(k, dy, dh)
    assert out["y"].shape == (0, 5, 8) and not out["da"].any() and not out["dd"].any() and not out["ddt_bias"].any()
    k, dy, dh = inputs(2, 0, 8, 4, 1, f32)
    out = run(k, dy, dh)
    assert torch.equal(out["h"], k["h0"]) and torch.equal(out["dh0"], dh) and not out["da"].any()
    h = torch.zeros(0, 8, 4, device="cuda")
    assert ssm.ssm_scan_step(h, *[k[m][:0, 0] if m in ROWS else k[m] for m in ()], torch.zeros(0, 8, device="cuda"), torch.zeros(0, 8, device="cuda"),
                             k["a"], torch.zeros(0, 1, 4, device="cuda"), torch.zeros(0, 1, 4, device="cuda")).shape == (0, 8)


def test_repeats_streams_and_graphs():
    """Bitwise the same run to run, on another stream, and replayed with other inputs."""
    say("[ssm] repeats, streams, graphs")
    kw = dict(reset=flags(2, 300, 3, 0.01))
    k, dy, dh = inputs(2, 300, 100, 16, 1, bf, seed=20)
    first = run(k, dy, dh, **kw)
    again = run(k, dy, dh, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(k, dy, dh, **kw, stream=side)
    for n in first:
        assert torch.equal(first[n], again[n]) and torch.equal(first[n], other[n]), n
    graph = torch.cuda.CUDAGraph()
    args = [k[n] for n in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")]
    with torch.cuda.graph(graph):
        y, h, saved = ssm.ssm_scan_fwd(*args, k["h0"], **kw)
        out = dict(y=y, h=h, **ssm.ssm_scan_bwd(*args, saved, dy, dh, want_dh0=True, **kw))
    for seed in (21, 22, 23):
        m, my, mh = inputs(2, 300, 100, 16, 1, bf, seed=seed)
        want = run(m, my, mh, **kw)
        for n in k:
            k[n].copy_(m[n])
        dy.copy_(my)
        dh.copy_(mh)
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]), (seed, n)


def test_step_in_a_graph():
    say("[ssm] step in a graph")
    k, _, _ = inputs(4, 1, 64, 16, 1, bf, seed=30)
    args = [k[n] if n in ("a", "d", "dt_bias") else k[n][:, 0] for n in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")]
    h, eager = k["h0"].clone(), k["h0"].clone()
    ssm.ssm_scan_step(h.clone(), *args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ssm.ssm_scan_step(h, *args)
    for i in range(4):
        k["u"].normal_()
        want = ssm.ssm_scan_step(eager, *args)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(h, eager), i


def test_gradients_against_differences():
    """Along a direction v: (f(x + v) - f(x - v)) / 2, with v a 64th of the input's size and the sums in 64 bits.  How far that is from the slope
    itself, the function bending, is taken from the definition in 64 bits (a sixth of the third derivative along v: of a, whose gradient
    is largest where a is smallest, it is a fifth of the slope); the outputs' roundings are below a hundredth."""
    say("[ssm] differences")
    k, dy, dh = inputs(2, 40, 24, 8, 2, f32, seed=40, scale=0.5)
    g = run(k, dy, dh)
    exact = scan_ref(**k, dy=dy, dh_final=dh)

    def loss(r):
        return float((r["y"].double() * dy.double()).sum() + (r["h"].double() * dh.double()).sum())

    names = dict(u="du", dt="ddt", a="da", b="db", c="dc", d="dd", z="dz", dt_bias="ddt_bias", h0="dh0")
    for n, name in names.items():
        v = g[name] * (k[n].norm() / g[name].norm() / 64)       # along the gradient
        more, less = {**k, n: k[n] + v}, {**k, n: k[n] - v}
        diff = (loss(run(more, None, None)) - loss(run(less, None, None))) / 2
        bend = (loss(scan_ref(**more)) - loss(scan_ref(**less))) / 2 - float((exact[name] * v.double()).sum())
        along = float((g[name].double() * v.double()).sum())
        assert abs(diff - bend - along) < 0.01 * along, (n, diff, bend, along)


def test_autograd():
    say("[ssm] autograd")
    k, dy, dh = inputs(2, 30, 20, 16, 1, bf, seed=50)
    kw = dict(reset=flags(2, 30, 1))
    want = run(k, dy, dh, **kw)
    leaf = {n: t.clone().requires_grad_() for n, t in k.items()}
    y, h = autograd.ssm_scan(**leaf, **kw)
    assert torch.equal(y, want["y"]) and torch.equal(h, want["h"])
    got = torch.autograd.grad([y, h], list(leaf.values()), [dy, dh], retain_graph=True)
    names = dict(u="du", dt="ddt", a="da", b="db", c="dc", d="dd", z="dz", dt_bias="ddt_bias", h0="dh0")
    for n, t in zip(leaf, got):
        assert torch.equal(t, want[names[n]]), n
    only = torch.autograd.grad(y.float().sum(), [leaf["u"]], retain_graph=True)[0]     # an expanded cotangent, none of the state
    assert torch.equal(only, run(k, torch.ones_like(dy), None, **kw)["du"])
    only = torch.autograd.grad(h.sum(), [leaf["a"]], retain_graph=True)[0]
    assert torch.equal(only, run(k, torch.zeros_like(dy), torch.ones_like(dh), **kw)["da"])
    with pytest.raises(RuntimeError, match="no second derivative"):
        torch.autograd.grad(torch.autograd.grad(y.float().sum(), [leaf["u"]], create_graph=True)[0].sum(), [leaf["b"]])
    with torch.no_grad():
        y2, h2 = autograd.ssm_scan(**leaf, **kw)
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_written_outputs_count_as_modified():
    say("[ssm] versions")
    k, _, _ = inputs(2, 5, 8, 4, 1, f32, seed=60)
    args = [k[n] for n in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")]
    y, h = torch.empty_like(k["u"]), torch.empty_like(k["h0"])
    r = ssm.ssm_scan_fwd(*args, y=y, h_final=h, want_saved=False)
    assert r[0] is y and r[1] is h and r[2] is None and y._version == 1 and h._version == 1
    state = k["h0"].clone()
    v = state._version
    ssm.ssm_scan_step(state, *[k[n] if n in ("a", "d", "dt_bias") else k[n][:, 0] for n in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")])
    assert state._version == v + 1
