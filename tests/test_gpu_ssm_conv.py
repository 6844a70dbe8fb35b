"""The short causal convolution on the GPU against its definition in 64 bits."""
import pytest
import torch

from linear_recurrence_sequence_amd import autograd, ssm
from tests.helpers import say
from tests.ssm_ref import U, conv_ref, half_step

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def inputs(batch, length, d, width, dtype, seed=0, full=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dt=f32):
        return torch.randn(shape, generator=g, device="cuda").to(dt)

    k = dict(x=normal(batch, length, d, dt=dtype), w=normal(d, width), bias=normal(d) if full else None,
             state=normal(batch, width - 1, d, dt=dtype) if full else None)
    return k, normal(batch, length, d, dt=dtype), normal(batch, width - 1, d, dt=dtype) if full else None


def run(k, dy, do, act="silu", **kw):
    y, last = ssm.causal_conv_fwd(k["x"], k["w"], k["bias"], act=act, state=k["state"], **kw)
    out = dict(y=y, last=last)
    if dy is not None:
        out.update(ssm.causal_conv_bwd(k["x"], k["w"], k["bias"], dy, do, act=act, state=k["state"], **kw))
    torch.cuda.synchronize()
    return out


def check(got, k, dy, do, act, kw, dtype):
    """p takes width multiply-adds (at most 4 halves of a step, relative to the sizes added up), its sigmoid 4, the slope 6 and the products
    with it 3; dx adds 4 more; sums over tokens are FP32 over at most 64 of a piece, FP64 from there: with 100 halves of a step all
    of it is covered.  A result of `dtype` is rounded once more; inputs handed on are exact."""
    ref = conv_ref(**k, silu=act == "silu", **kw, dy=dy, dstate_out=do)
    size = conv_ref(**k, silu=act == "silu", **kw, dy=dy, dstate_out=do, absolute=True)
    for n, t in got.items():
        tol = 100 * U * size[n] + (half_step(dtype) * ref[n].abs() if n not in ("dw", "dbias") else 0.0) + 1e-37
        if n == "last":
            tol = torch.zeros_like(ref[n])
        err = (t.double() - ref[n]).abs()
        assert t.shape == ref[n].shape and t.dtype == (f32 if n in ("dw", "dbias") else dtype)
        assert (err <= tol).all(), (n, float(err.max()), int((~(err <= tol)).sum()))


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("batch,length,d,width", [(1, 1, 1, 2), (2, 1, 3, 4), (1, 2, 4, 4), (2, 3, 5, 4), (1, 8, 64, 3), (3, 9, 65, 2), (2, 66, 30, 4),
                                                  (1, 200, 257, 4), (2, 37, 1026, 3)])
def test_parity(dtype, act, batch, length, d, width):
    say(f"[conv] {dtype} {act} batch={batch} length={length} d={d} width={width}")
    for full in (True, False):
        k, dy, do = inputs(batch, length, d, width, dtype, seed=length, full=full)
        check(run(k, dy, do, act), k, dy, do, act, {}, dtype)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("length", [1, 2, 5, 40, 150])
def test_packed_and_padded(dtype, width, length):
    say(f"[conv] packed and padded {dtype} width={width} length={length}")
    k, dy, do = inputs(3, length, 11, width, dtype, seed=length)
    g = torch.Generator(device="cuda").manual_seed(width)
    reset = (torch.rand(3, length, generator=g, device="cuda") < 0.3).to(torch.uint8)
    lengths = torch.tensor([length // 2, length, 0], dtype=torch.int32, device="cuda")
    for kw in (dict(reset=reset), dict(lengths=lengths), dict(reset=reset.bool(), lengths=lengths),
               dict(lengths=torch.tensor([-2, length + 5, 1], dtype=torch.int32, device="cuda")),
               dict(reset=torch.ones(3, length, dtype=torch.uint8, device="cuda"))):
        check(run(k, dy, do, **kw), k, dy, do, "silu", kw, dtype)


def test_nothing_crosses_a_start_or_comes_from_padding():
    say("[conv] NaN before a start and in padding")
    k, dy, do = inputs(2, 150, 12, 4, bf, seed=2)
    reset = torch.zeros(2, 150, dtype=torch.uint8, device="cuda")
    reset[:, 30] = 1
    kw = dict(reset=reset, lengths=torch.tensor([100, 140], dtype=torch.int32, device="cuda"))
    want = run(k, dy, do, **kw)
    for bad in (float("nan"), float("inf")):
        p, py = {n: t.clone() for n, t in k.items()}, dy.clone()
        for i, end in enumerate((100, 140)):
            p["x"][i, end:] = bad
            py[i, end:] = bad
        got = run(p, py, do, **kw)
        for n in want:
            assert torch.equal(got[n], want[n]), n
        p["x"][:, 29] = bad
        p["state"][:] = bad
        got = run(p, py, do, **kw)
        assert torch.equal(got["y"][:, 30:], want["y"][:, 30:]) and torch.equal(got["dx"][:, 30:], want["dx"][:, 30:])
        assert torch.equal(got["last"], want["last"])
        py = torch.where(py.isfinite(), py, dy)
        py[:, 31] = bad
        got = run(k, py, do, **kw)
        assert torch.equal(got["dx"][:, :30], want["dx"][:, :30]) and torch.equal(got["dstate"], want["dstate"])


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_rows_that_lie_apart(dtype):
    say(f"[conv] strides {dtype}")
    k, dy, do = inputs(2, 21, 18, 4, dtype, seed=4)
    want = run(k, dy, do)
    buf = torch.full((2, 21, 41), float("nan"), dtype=dtype, device="cuda")
    buf[..., 1:19], buf[..., 20:38] = k["x"], dy
    got = run({**k, "x": buf[..., 1:19]}, buf[..., 20:38], do)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("batch,d,width", [(1, 1, 4), (3, 66, 4), (2, 301, 3), (5, 64, 2)])
def test_step(dtype, act, batch, d, width):
    """Token by token as the whole row: the same roundings, so the same bits."""
    say(f"[conv] step {dtype} {act} batch={batch} d={d} width={width}")
    k, _, _ = inputs(batch, 7, d, width, dtype, seed=5)
    want = run(k, None, None, act)
    state = k["state"].clone()
    for t in range(7):
        y = ssm.causal_conv_step(k["x"][:, t], k["w"], k["bias"], state, act=act)
        assert torch.equal(y, want["y"][:, t])
    assert torch.equal(state, want["last"])


def test_empty():
    say("[conv] nothing to do")
    k, dy, do = inputs(0, 4, 8, 4, f32)
    out = run(k, dy, do)
    assert out["y"].shape == (0, 4, 8) and not out["dw"].any() and not out["dbias"].any()
    k, dy, do = inputs(2, 0, 8, 4, f32)
    out = run(k, dy, do)
    assert torch.equal(out["last"], k["state"]) and torch.equal(out["dstate"], do) and not out["dw"].any()


def test_repeats_streams_and_graphs():
    say("[conv] repeats, streams, graphs")
    k, dy, do = inputs(2, 300, 100, 4, bf, seed=20)
    first = run(k, dy, do)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(k, dy, do, stream=side)
    for n in first:
        assert torch.equal(first[n], other[n]), n
    graph = torch.cuda.CUDAGraph()
    state = k["state"].clone()
    with torch.cuda.graph(graph):
        y, last = ssm.causal_conv_fwd(k["x"], k["w"], k["bias"], state=k["state"])
        out = dict(y=y, last=last, **ssm.causal_conv_bwd(k["x"], k["w"], k["bias"], dy, do, state=k["state"]))
        moved = ssm.causal_conv_step(k["x"][:, 0], k["w"], k["bias"], state)
    eager = k["state"].clone()
    for seed in (21, 22, 23):
        m, my, mo = inputs(2, 300, 100, 4, bf, seed=seed)
        want = run(m, my, mo)
        for n in k:
            k[n].copy_(m[n])
        dy.copy_(my)
        do.copy_(mo)
        one = ssm.causal_conv_step(k["x"][:, 0], k["w"], k["bias"], eager)
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]), (seed, n)
        assert torch.equal(moved, one) and torch.equal(state, eager)


def test_autograd():
    say("[conv] autograd")
    k, dy, do = inputs(2, 30, 20, 4, bf, seed=50)
    want = run(k, dy, do)
    leaf = {n: t.clone().requires_grad_() for n, t in k.items()}
    y, last = autograd.causal_conv(leaf["x"], leaf["w"], leaf["bias"], leaf["state"])
    assert torch.equal(y, want["y"]) and torch.equal(last, want["last"])
    got = torch.autograd.grad([y, last], list(leaf.values()), [dy, do], retain_graph=True)
    for n, t in zip(("dx", "dw", "dbias", "dstate"), got):
        assert torch.equal(t, want[n]), n
    only = torch.autograd.grad(last.float().sum(), [leaf["x"]], retain_graph=True)[0]
    assert torch.equal(only, run(k, torch.zeros_like(dy), torch.ones_like(do))["dx"])
    with pytest.raises(RuntimeError, match="no second derivative"):
        torch.autograd.grad(torch.autograd.grad(y.float().sum(), [leaf["x"]], create_graph=True)[0].sum(), [leaf["w"]])


def test_gradients_against_differences():
    """As for the scan: a hundredth covers the third derivative and FP32's roundings, with steps of a 64th of an input."""
    say("[conv] differences")
    k, dy, do = inputs(2, 40, 24, 4, f32, seed=40)
    g = run(k, dy, do)

    def loss(m):
        r = run(m, None, None)
        return float((r["y"].double() * dy.double()).sum() + (r["last"].double() * do.double()).sum())

    for n, name in dict(x="dx", w="dw", bias="dbias", state="dstate").items():
        v = g[name] * (k[n].norm() / g[name].norm() / 64)
        diff = (loss({**k, n: k[n] + v}) - loss({**k, n: k[n] - v})) / 2
        along = float((g[name].double() * v.double()).sum())
        assert abs(diff - along) < 0.01 * along, (n, diff, along)
