"""The embedding lookup and its gradient on the GPU against their definitions in 64 bits."""
import pytest
import torch

from linear_recurrence_sequence_amd import autograd, lm
from tests.helpers import say
from tests.ssm_ref import U, embed_ref, half_step

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def tokens_of(kind, n, v, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":
        return torch.full((n,), v // 2, device="cuda")
    if kind == "few":                                  # rows with many tokens each, next to each other in the order
        return torch.randint(0, min(v, 7), (n,), generator=g, device="cuda")
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    if kind == "mixed":                                # one row has a third, some are padding, some beyond the vocabulary
        r = torch.rand(n, generator=g, device="cuda")
        t = torch.where(r < 0.33, torch.full_like(t, v - 1), t)
        t = torch.where(r > 0.9, torch.full_like(t, -1), t)
        t = torch.where(r > 0.95, torch.full_like(t, -100), t)
        t = torch.where(r > 0.98, torch.full_like(t, v + 3), t)
    return t


@pytest.mark.parametrize("wt", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ot", [bf, f32], ids=["to_bf16", "to_f32"])
@pytest.mark.parametrize("n,d,v", [(1, 1, 1), (3, 5, 7), (16, 64, 100), (70, 257, 513), (5, 1030, 20)])
def test_lookup(wt, ot, n, d, v):
    """One product, rounded: half a step of FP32, then of the result."""
    say(f"[embed] {wt} {ot} n={n} d={d} v={v}")
    w = torch.randn(v, d, device="cuda").to(wt)
    t = tokens_of("uniform", n, v)
    got = lm.embed_fwd(t, w, scale=1.7, out_dtype=ot)
    want = w[t].double() * 1.7
    assert got.dtype == ot and ((got.double() - want).abs() <= (2 * U + half_step(ot)) * want.abs()).all()
    assert torch.equal(lm.embed_fwd(t, w), w[t])
    t[0] = -1
    got = lm.embed_fwd(t.reshape(1, n), w, out_dtype=ot)
    assert got.shape == (1, n, d) and not got[0, 0].any()
    t[-1] = v
    assert lm.embed_fwd(t, w, out_dtype=ot)[-1].isnan().all()


@pytest.mark.parametrize("ot", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gt", [bf, f32], ids=["to_bf16", "to_f32"])
@pytest.mark.parametrize("kind", ["uniform", "one", "few", "mixed"])
@pytest.mark.parametrize("n,d,v", [(1, 4, 1), (31, 6, 9), (33, 64, 40), (64, 7, 600), (700, 260, 1500), (3000, 33, 513), (2500, 1, 5000)])
def test_gradient(ot, gt, kind, n, d, v):
    """A sum of k values in FP32 is off by less than k halves of a step of their sizes' sum, the scale takes one more."""
    say(f"[embed] gradient {ot} {gt} {kind} n={n} d={d} v={v}")
    t = tokens_of(kind, n, v, seed=n)
    dout = torch.randn(n, d, generator=torch.Generator(device="cuda").manual_seed(d), device="cuda").to(ot)
    got = lm.embed_bwd(t, dout, v, scale=0.3, grad_dtype=gt)
    want, size = embed_ref(t, dout, v, 0.3), embed_ref(t, dout, v, 0.3, absolute=True)
    most = int(torch.bincount(t[(t >= 0) & (t < v)], minlength=v).max())
    assert got.dtype == gt and ((got.double() - want).abs() <= (most + 2) * U * size + half_step(gt) * want.abs()).all()
    base = torch.randn(v, d, device="cuda").to(gt)
    dw = base.clone()
    assert lm.embed_bwd(t, dout, v, scale=0.3, dw=dw, accumulate=True) is dw
    total = base.double() + want
    assert ((dw.double() - total).abs() <= (most + 3) * U * (size + base.double().abs()) + half_step(gt) * total.abs()).all()
    empty = torch.bincount(t[(t >= 0) & (t < v)], minlength=v) == 0
    assert torch.equal(dw[empty], base[empty]) and not got[empty].any()


def test_order_is_that_of_the_tokens():
    """Sums whose value depends on their order: the same bits whatever the schedule, and those of the order where a row has few tokens."""
    say("[embed] order")
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.randint(0, 300, (9000,), generator=g, device="cuda")
    dout = torch.randn(9000, 40, generator=g, device="cuda") * torch.exp(4 * torch.randn(9000, 1, generator=g, device="cuda"))
    first = lm.embed_bwd(t, dout, 300, grad_dtype=f32)
    for _ in range(3):
        assert torch.equal(first, lm.embed_bwd(t, dout, 300, grad_dtype=f32))
    few = torch.randint(0, 300, (900,), generator=g, device="cuda")
    got, want = lm.embed_bwd(few, dout[:900], 300, grad_dtype=f32).cpu(), torch.zeros(300, 40)
    counts = torch.bincount(few, minlength=300)
    for i, j in enumerate(few.tolist()):
        want[j] += dout[i].cpu()
    rows = (counts <= 32).cpu()
    assert rows.any() and torch.equal(got[rows], want[rows])


def test_strides_and_padding():
    say("[embed] strides, padding")
    t = tokens_of("mixed", 200, 50)
    buf = torch.full((200, 75), float("nan"), device="cuda")
    buf[:, 2:72] = torch.randn(200, 70, device="cuda")
    dout = buf[:, 2:72]
    want = lm.embed_bwd(t, dout.contiguous(), 50, grad_dtype=f32)
    assert torch.equal(lm.embed_bwd(t, dout, 50, grad_dtype=f32), want)
    out = (t < 0) | (t >= 50)
    dout[out] = float("nan")                           # what stands for tokens that have no gradient is not read into any
    assert torch.equal(lm.embed_bwd(t, dout, 50, grad_dtype=f32), want)
    none = torch.full((100,), -1, device="cuda")
    assert not lm.embed_bwd(none, torch.randn(100, 70, device="cuda"), 50).any()
    assert not lm.embed_bwd(none[:0], torch.randn(0, 70, device="cuda"), 50).any()
    dw = torch.ones(50, 70, device="cuda")
    assert torch.equal(lm.embed_bwd(none[:0], torch.randn(0, 70, device="cuda"), 50, dw=dw, accumulate=True), torch.ones_like(dw))
    assert lm.embed_fwd(none[:0], dw).shape == (0, 70)
    one = torch.randn(1, 70, device="cuda").expand(200, 70)
    assert torch.equal(lm.embed_bwd(t, one, 50), lm.embed_bwd(t, one.contiguous(), 50))


def test_streams_and_graphs():
    say("[embed] streams, graphs")
    t, w = tokens_of("mixed", 500, 90), torch.randn(90, 30, device="cuda").to(bf)
    dout = torch.randn(500, 30, device="cuda").to(bf)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = lm.embed_fwd(t, w, stream=side), lm.embed_bwd(t, dout, 90, stream=side)
    side.synchronize()
    assert torch.equal(a.nan_to_num(), lm.embed_fwd(t, w).nan_to_num()) and torch.equal(b, lm.embed_bwd(t, dout, 90))
    graph = torch.cuda.CUDAGraph()
    dw = torch.zeros(90, 30, device="cuda")
    with torch.cuda.graph(graph):
        out, grad = lm.embed_fwd(t, w), lm.embed_bwd(t, dout, 90)
        lm.embed_bwd(t, dout, 90, dw=dw, accumulate=True)
    dw.zero_()
    eager = torch.zeros_like(dw)
    for seed in range(3):
        t.copy_(tokens_of("uniform", 500, 90, seed))
        dout.normal_()
        want = lm.embed_fwd(t, w), lm.embed_bwd(t, dout, 90)
        lm.embed_bwd(t, dout, 90, dw=eager, accumulate=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(grad, want[1]) and torch.equal(dw, eager)


def test_autograd():
    say("[embed] autograd")
    t = tokens_of("mixed", 60, 40).clamp_max(39).reshape(3, 20)
    w = torch.randn(40, 24, device="cuda").to(bf).requires_grad_()
    out = autograd.embed(t, w, scale=2.0, out_dtype=f32)
    assert torch.equal(out, lm.embed_fwd(t, w, scale=2.0, out_dtype=f32))
    dout = torch.randn_like(out)
    g = torch.autograd.grad(out, [w], [dout], retain_graph=True)[0]
    assert g.dtype == bf and torch.equal(g, lm.embed_bwd(t, dout, 40, scale=2.0))
    assert torch.equal(torch.autograd.grad(out.sum(), [w], retain_graph=True)[0], lm.embed_bwd(t, torch.ones_like(dout), 40, scale=2.0))
    x = torch.ones_like(out).requires_grad_()
    with pytest.raises(RuntimeError, match="no second derivative"):
        torch.autograd.grad(torch.autograd.grad((out * x).sum(), [w], create_graph=True)[0].float().sum(), [x])
    v = out._version
    lm.embed_fwd(t, w.detach(), out=out.detach(), out_dtype=f32)
    assert out._version == v + 1
