"""The selective scan over rows that are cut into segments: what is handed from one to the next."""
import pytest
import torch

from linear_recurrence_sequence_amd import ssm
from tests.helpers import say
from tests.ssm_ref import scan_ref, scan_tolerance
from tests.test_gpu_ssm_scan import check, inputs, run

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def segments_of(batch, length, width, n, groups):
    """Segments of a row in the forward: its workspace holds two records of [n, width] for each, where there are several."""
    size = ssm.lib().ssm_scan_workspace_bytes(batch, length, width, n, groups, 0)
    return max(1, size // (batch * 2 * n * width * 4))


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_what_is_not_finite_stays(dtype, bad):
    """A state that is not finite stays so to its sequence's end, a cotangent to its start, however much the decays between are: a
    segment's product of them here is below what FP32 holds."""
    say(f"[ssm] not finite, {dtype} {bad}")
    batch, length, width, n = 1, 2000, 40, 8
    assert segments_of(batch, length, width, n, 1) > 30
    k, dy, dh = inputs(batch, length, width, n, 1, dtype, seed=31)
    k["a"] = -torch.rand(width, n, device="cuda") - 3
    k["dt_bias"] += 4                                            # steps around two: decays of e^-6 a token
    kw = dict(reset=torch.zeros(batch, length, dtype=torch.uint8, device="cuda"))
    kw["reset"][:, 1500] = 1
    clean = run(k, dy, dh, **kw)
    m = {x: t.clone() for x, t in k.items()}
    m["u"][0, 5, 3] = bad
    got, ref = run(m, None, None, **kw), scan_ref(**m, **kw)
    assert not got["y"][0, 5:1500, 3].isfinite().any() and torch.equal(got["y"].isfinite(), ref["y"].isfinite())
    assert torch.equal(got["h"], clean["h"])
    late = dy.clone()
    late[0, 1400, 3] = bad
    got = run(k, late, dh, **kw)
    assert not got["du"][0, :1401, 3].isfinite().any() and not got["ddt"][0, :1400, 3].isfinite().any() and not got["dh0"][0, 3].isfinite().any()
    others = [i for i in range(width) if i != 3]
    for name in ("du", "ddt", "dz"):
        assert torch.equal(got[name][:, 1401:], clean[name][:, 1401:]) and torch.equal(got[name][..., others], clean[name][..., others]), name
    kw["reset"][:] = 0
    m["u"][0, 5, 3] = 0.5
    m["h0"][0, 3, 2] = bad
    got = run(m, None, None, **kw)
    assert not got["y"][0, :, 3].isfinite().any() and not got["h"][0, 3, 2].isfinite().any() and got["y"][0, :, others].isfinite().all()


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_growing_decays_of_nothing(dtype):
    """Steps may be negative where softplus is off: products of a segment's factors are then beyond FP32.  States that are zero, and
    cotangents that are, stay so."""
    say(f"[ssm] growth of nothing, {dtype}")
    batch, length, width, n = 1, 2000, 40, 8
    assert segments_of(batch, length, width, n, 1) > 30
    k, dy, _ = inputs(batch, length, width, n, 1, dtype, seed=32, full=False)
    k["a"] = -torch.rand(width, n, device="cuda") - 3
    k["dt"] = k["dt"].abs() * 0.1 + 0.05
    k["dt"][:, :800] = -1.0                                     # factors of e^3 to e^4 a token, of states that no input has reached
    k["u"][:, :800] = 0
    k["dt"][:, 1300:] = -1.0                                    # and of cotangents that no output has
    k["u"][:, 1300:] = 0
    dy[:, 1300:] = 0
    kw = dict(softplus=False, reset=torch.zeros(batch, length, dtype=torch.uint8, device="cuda"))
    kw["reset"][:, 1300] = 1
    got = run(k, dy, None, **kw)
    check({x: got[x] for x in ("y", "h")}, k, dy, None, kw, dtype, length)
    assert not got["y"][:, :800].any() and not got["du"][:, 1300:].any()
    # before the 800th token cotangents grow by e^3 a token: there the definition's own are beyond FP32, and beyond 64 bits further up
    ref, size = scan_ref(**k, **kw, dy=dy), scan_ref(**k, **kw, dy=dy, absolute=True)
    tol = scan_tolerance(size, ref, length, dtype)
    for x in ("du", "ddt", "dz", "db", "dc"):
        assert ((got[x].double() - ref[x]).abs() <= tol[x])[:, 800:].all(), x


def test_growth_beyond_fp32_of_small_states():
    """A segment whose product of factors is about 2^138, of a state small enough that nothing overflows, and one of 2^-200 of a large state."""
    say("[ssm] growth of small states")
    batch, length, width, n = 1, 2000, 40, 8
    segments = segments_of(batch, length, width, n, 1)
    assert segments > 30
    k, dy, dh = inputs(batch, length, width, n, 1, f32, seed=33)
    part = -(-125 // segments) * 16                              # tokens of a segment
    k["dt_bias"] = None
    k["d"] = None
    k["a"] = torch.full((width, n), -3.0, device="cuda")
    k["dt"] = torch.full_like(k["dt"], 1e-3)
    k["dt"][:, 4 * part:5 * part] = -138 * 0.6931 / 3 / part
    k["dt"][:, 8 * part:9 * part] = 200 * 0.6931 / 3 / part
    k["u"] *= 1e-25
    k["h0"] *= 1e-25
    k["u"][:, 4 * part:5 * part] = 0
    k["u"][:, 8 * part:] = 0
    dy *= 1e-10
    dh *= 1e-10
    kw = dict(softplus=False)
    check(run(k, dy, dh, **kw), k, dy, dh, kw, f32, length)
