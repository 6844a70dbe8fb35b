"""The selective scan over rows that are cut into segments: what is handed from one to the next."""
import pytest
import torch

from linear_recurrence_sequence_amd import ssm
from tests.helpers import say
from tests.ssm_ref import scan_ref
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
