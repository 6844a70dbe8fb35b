"""Linear cross entropy on the GPU against the definition in 64 bits.

Tolerances, element by element.  A logit is an FP32 sum of exact BF16 products:
off by at most e_z = 2e-6 of its sum of magnitudes (a few dozen roundings of
2^-24 each), plus 4e-7 of the cap where there is one.  lse and the target's
logit are each off by the largest e_z of the token and 1e-6 of their value.
Backward, dz is rounded to BF16 (2^-8 of the term) and exp carries e_z: dh is
off by (2^-8 + 2 e_z + 1e-5) of its sum of magnitudes, plus 2^-8 of itself where
it is BF16.  The same holds for dw."""
import pytest
import torch

from linear_recurrence_sequence_amd import autograd, lm
from tests.helpers import say

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def make(n, d, v, seed, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    w = r(v, d) * (std / d ** 0.5)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    h = r(n, d) + (3.0 * torch.rand(n, 1, generator=g, device="cuda") * w[t] if n else 0.0)
    t = torch.where(torch.rand(n, generator=g, device="cuda") < 0.2, torch.full_like(t, -100), t)
    return dict(h=h.to(bf), w=w.to(bf), t=t, dloss=r(n).abs() / max(n, 1), dlse=1e-2 * r(n) / max(n, 1))


def exact(a, cap, dlse):
    h, w, t = a["h"].double(), a["w"].double(), a["t"]
    z = h @ w.t()
    ez = 2e-6 * (h.abs() @ w.abs().t()).amax(1) + 4e-7 * cap
    slope = torch.ones_like(z)
    if cap:
        th = torch.tanh(z / cap)
        z, slope = cap * th, 1 - th * th
    lse = torch.logsumexp(z, 1)
    on = t >= 0
    row = torch.arange(len(t), device="cuda")
    picked = z[row, t.clamp_min(0)]
    loss = torch.where(on, lse - picked, torch.zeros_like(lse))
    dl = torch.where(on, a["dloss"].double(), torch.zeros_like(lse))
    c = dl if dlse is None else dl + dlse.double()
    dz = torch.exp(z - lse[:, None]) * c[:, None]
    mag = dz.abs()
    dz[row, t.clamp_min(0)] -= dl
    mag[row, t.clamp_min(0)] += dl
    dz, mag = dz * slope, mag * slope
    rel = 2.0 ** -8 + 2 * float(ez.max() if len(t) else 0) + 1e-5
    return dict(lse=lse, loss=loss, ez=ez, picked=picked, dh=dz @ w, dw=dz.t().contiguous() @ h,
                tol_h=rel * (mag @ w.abs()), tol_w=rel * (mag.t().contiguous() @ h.abs()))


def within(got, ref, tol, what):
    if got.dtype == bf:
        tol = tol + 2.0 ** -8 * ref.abs()
    bad = (got.double() - ref).abs() - tol - 2.0 ** -126
    assert not got.numel() or float(bad.max()) <= 0, (what, float(bad.max()), float((got.double() - ref).abs().max()))


def check(a, cap=0.0, zloss=False, grad_dtype=bf, backward=True):
    dlse = a["dlse"] if zloss else None
    ref = exact(a, cap, dlse)
    loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"], softcap=cap)
    within(lse, ref["lse"], ref["ez"] + 1e-6 * ref["lse"].abs(), "lse")
    within(loss, ref["loss"], 2 * ref["ez"] + 1e-6 * (ref["lse"].abs() + ref["picked"].abs()), "loss")
    if backward:
        g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"], dlse, softcap=cap, grad_dtype=grad_dtype)
        assert g["dh"].dtype == grad_dtype
        within(g["dh"], ref["dh"], ref["tol_h"], "dh")
        within(g["dw"], ref["dw"], ref["tol_w"], "dw")


@pytest.mark.parametrize("n,d,v", [(1, 8, 1), (1, 64, 7), (2, 24, 64), (16, 1024, 4000), (15, 72, 257), (32, 136, 1000), (33, 8, 63),
                                   (40, 200, 65), (128, 128, 128), (129, 264, 129), (300, 520, 999), (257, 64, 5000), (100, 2048, 300)])
def test_shapes(n, d, v):
    say(f"[ce] n={n} d={d} v={v}")
    a = make(n, d, v, 1000 * n + d + v)
    check(a, cap=30.0 if n % 2 else 0.0, zloss=bool(d % 16), grad_dtype=f32 if v % 2 else bf)


@pytest.mark.parametrize("n,d,v", [(512, 64, 25001), (520, 96, 25000), (2048, 8192, 300), (2050, 6160, 520)])
def test_many_tiles(n, d, v):
    say(f"[ce] many tiles n={n} d={d} v={v}")
    check(make(n, d, v, n + d), cap=0.0, zloss=True)


def test_vocabulary_in_several_chunks():
    say("[ce] several chunks")
    n, d, v = 8200, 64, 20001
    assert lm.lib().lm_linear_ce_workspace_bytes(n, d, v, 1) < n * v * 2
    check(make(n, d, v, 3), cap=0.0, zloss=True)


@pytest.mark.parametrize("cap", [0.0, 5.0, 30.0])
@pytest.mark.parametrize("zloss", [False, True])
def test_forms(cap, zloss):
    for n, d, v in ((20, 64, 300), (200, 64, 700)):
        say(f"[ce] cap={cap} zloss={zloss} n={n}")
        check(make(n, d, v, 7, std=6.0), cap=cap, zloss=zloss)


def test_no_token_counts():
    say("[ce] every target negative")
    a = make(70, 64, 500, 8)
    a["t"].fill_(-1)
    loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])
    assert bool((loss == 0).all()) and bool(torch.isfinite(lse).all())
    a["dloss"].fill_(float("nan"))            # not read for a token that does not count
    g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"])
    assert bool((g["dh"] == 0).all()) and bool((g["dw"] == 0).all())


def test_no_tokens():
    say("[ce] zero tokens")
    a = make(0, 64, 77, 9)
    loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])
    assert loss.shape == (0,) and lse.shape == (0,)
    for dt in (bf, f32):
        dw = torch.ones(77, 64, dtype=dt, device="cuda")
        g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"], dw=dw, dh=torch.empty(0, 64, dtype=dt, device="cuda"))
        assert g["dh"].shape == (0, 64) and bool((dw == 0).all())


def test_target_beyond_the_vocabulary_and_a_bad_row():
    """NaN for the token whose target does not exist; a NaN row stays its own in loss and lse."""
    say("[ce] target out of range, NaN row")
    for n in (10, 200):
        a = make(n, 64, 300, 10)
        a["t"][3] = 300
        a["t"][4] = 1 << 40
        a["h"][6] = float("nan")
        a["t"][6] = -100
        loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])
        assert torch.isnan(loss).nonzero().reshape(-1).tolist() == [3, 4]
        assert torch.isnan(lse).nonzero().reshape(-1).tolist() == [6]
        g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"])
        rows = torch.isnan(g["dh"]).any(1).nonzero().reshape(-1).tolist()
        assert rows == [3, 4]
        assert bool((g["dh"][6] == 0).all())


def test_large_logits():
    """Logits of several hundred: exp of none of them overflows, and a certain token has loss zero."""
    say("[ce] large logits")
    for n in (8, 160):
        a = make(n, 64, 400, 11, std=200.0)
        a["h"] = (a["h"].float() * 4).to(bf)
        check(a)
        loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])
        assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(lse).all())


def test_strided_rows_guards_and_leading_dims():
    say("[ce] strided rows, guard values")
    n, d, v = 66, 72, 333
    a = make(n, d, v, 12)
    loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])
    g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"])
    wide = torch.full((n, d + 16), float("nan"), dtype=bf, device="cuda")
    wide[:, 8:8 + d] = a["h"]
    hs = wide[:, 8:8 + d]
    bufs = {k: torch.full((m + 256,), 7.0, dtype=t, device="cuda") for k, m, t in (("loss", n, f32), ("lse", n, f32), ("dh", n * d, bf), ("dw", v * d, bf))}

    def win(k, shape):
        return bufs[k][128:-128].view(shape)

    l2, e2 = lm.linear_ce_fwd(hs, a["w"], a["t"], loss=win("loss", (n,)), lse=win("lse", (n,)))
    lm.linear_ce_bwd(hs, a["w"], a["t"], e2, a["dloss"], dh=win("dh", (n, d)), dw=win("dw", (v, d)))
    assert torch.equal(l2, loss) and torch.equal(e2, lse)
    assert torch.equal(win("dh", (n, d)), g["dh"]) and torch.equal(win("dw", (v, d)), g["dw"])
    for b in bufs.values():
        assert bool((b[:128] == 7).all()) and bool((b[-128:] == 7).all())
    l3, _ = lm.linear_ce_fwd(a["h"].view(6, 11, d), a["w"], a["t"].view(6, 11))
    assert l3.shape == (6, 11) and torch.equal(l3.view(-1), loss)


def test_workspace_contents_do_not_matter():
    say("[ce] workspaces full of NaN")
    for n, d, v in ((7, 40, 1000), (150, 72, 777)):
        a = make(n, d, v, 13)
        def ws(b):
            return torch.full((lm.lib().lm_linear_ce_workspace_bytes(n, d, v, b) // 4,), float("nan"), device="cuda").view(torch.uint8)
        loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])
        g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"], a["dlse"])
        l2, e2 = lm.linear_ce_fwd(a["h"], a["w"], a["t"], workspace=ws(0))
        g2 = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"], a["dlse"], workspace=ws(1))
        assert torch.equal(loss, l2) and torch.equal(lse, e2)
        assert torch.equal(g["dh"], g2["dh"]) and torch.equal(g["dw"], g2["dw"])


def test_differences():
    """dh against central differences of the loss along random directions (BF16 steps that are exact)."""
    say("[ce] differences")
    n, d, v = 12, 64, 200
    a = make(n, d, v, 14)
    a["t"].clamp_(min=0)
    loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])
    g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"], grad_dtype=f32)
    e = torch.where(torch.rand(n, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) < 0.5, -1.0, 1.0)
    up, down = (a["h"].float() + e / 16).to(bf), (a["h"].float() - e / 16).to(bf)
    step = up.double() - down.double()
    f = [lm.linear_ce_fwd(h, a["w"], a["t"])[0].double() * a["dloss"].double() for h in (up, down)]
    got = (f[0] - f[1])
    mid = ((up.double() + down.double()) / 2 - a["h"].double())
    assert float(mid.abs().max()) < 0.05
    want = (g["dh"].double() * step).sum(1)
    # the step is ~1/8 along 64 columns, weights of 0.25 each: logits move by ~0.25, so third-order terms are a few per cent
    # of the token's weight, and rounding of h shifts the centre
    assert bool(((got - want).abs() <= 0.1 * a["dloss"].double()).all())


def test_autograd_stream_and_graph():
    say("[ce] autograd, side stream, graph")
    a = make(200, 96, 1234, 15)
    cap = 20.0
    loss, lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"], softcap=cap)
    want = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"], a["dlse"], softcap=cap)
    h, w = a["h"].clone().requires_grad_(), a["w"].clone().requires_grad_()
    l2, e2 = autograd.linear_ce(h, w, a["t"], softcap=cap)
    torch.autograd.backward([l2, e2], [a["dloss"], a["dlse"]])
    assert torch.equal(l2, loss) and torch.equal(h.grad, want["dh"]) and torch.equal(w.grad, want["dw"])
    l2, e2 = autograd.linear_ce(h, w, a["t"], softcap=cap)
    h.grad = None
    l2.sum().backward()                       # an expanded cotangent
    ones = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, torch.ones_like(lse), softcap=cap)
    assert torch.equal(h.grad, ones["dh"])
    del l2, e2
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def both():
        lo, ls = lm.linear_ce_fwd(a["h"], a["w"], a["t"], softcap=cap)
        return lo, ls, *lm.linear_ce_bwd(a["h"], a["w"], a["t"], ls, a["dloss"], a["dlse"], softcap=cap).values()

    with torch.cuda.stream(side):
        got = both()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = both()
    ref = (loss, lse, want["dh"], want["dw"])
    assert all(torch.equal(x, y) for x, y in zip(got, ref))
    for rep in range(3):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, ref)), rep
        both()


def test_rows_that_do_not_count_may_hold_anything():
    """NaN and infinite hidden rows of tokens that take no part reach neither gradient."""
    say("[ce] bad rows that do not count")
    for n, v in ((10, 300), (200, 300), (700, 1000)):
        a = make(n, 64, v, 16)
        good = {k: t.clone() for k, t in a.items()}
        a["t"][2::5] = -1
        good["t"][2::5] = -1
        a["h"][2::5] = float("nan")
        a["h"][2] = float("inf")
        lse = lm.linear_ce_fwd(good["h"], good["w"], good["t"])[1]
        want = lm.linear_ce_bwd(good["h"], good["w"], good["t"], lse, good["dloss"])
        lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])[1]
        got = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"])
        assert torch.equal(got["dh"], want["dh"]) and torch.equal(got["dw"], want["dw"])


@pytest.mark.parametrize("n,d,v", [(1500, 64, 700), (3000, 136, 260), (2200, 512, 2000)])
@pytest.mark.parametrize("kept", [0.0, 0.01, 0.5])
def test_most_tokens_do_not_count(n, d, v, kept):
    say(f"[ce] {kept} of the tokens count n={n}")
    a = make(n, d, v, 17)
    a["t"][torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) >= kept] = -100
    check(a, cap=20.0 if n % 4 else 0.0)


def test_weights_that_are_zero():
    """A token whose dloss is zero takes part through dlse alone, and one with neither gives exact zeros."""
    say("[ce] zero weights")
    a = make(300, 72, 500, 18)
    a["dloss"][::2] = 0.0
    a["dlse"][::3] = 0.0
    check(a, zloss=True)
    lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])[1]
    g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"], a["dlse"])
    assert bool((g["dh"][::6] == 0).all()) and bool((g["dh"][1::6] != 0).any(1).all())


def test_lists_longer_than_a_workgroup_pass():
    """More tokens than one pass of the listing workgroup, in one chunk and in several."""
    say("[ce] long lists")
    for n, d, v in ((5000, 64, 300), (9000, 64, 15000)):
        check(make(n, d, v, 19), zloss=n == 9000)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 65, 128, 129, 200, 256, 257])
@pytest.mark.parametrize("d,v", [(8, 17), (264, 700), (640, 5003)])
def test_few_tokens(n, d, v):
    """Around the counts where the layout of the few tokens' dz changes; some, one or no token with a weight."""
    say(f"[ce] few tokens n={n} d={d} v={v}")
    a = make(n, d, v, n + d)
    check(a, cap=15.0 if n % 3 == 0 else 0.0, zloss=n % 2 == 0, grad_dtype=f32 if v % 3 else bf)
    a["t"][: n - 1] = -1
    check(a)
    a["t"].fill_(-1)
    check(a)
