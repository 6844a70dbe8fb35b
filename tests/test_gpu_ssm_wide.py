"""The selective scan at its widest accepted sizes on the GPU."""
import pytest
import torch

from linear_recurrence_sequence_amd import ssm
from tests.helpers import say
from tests.ssm_ref import U, scan_ref, scan_tolerance

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def test_a_last_launch_of_more_than_2_32_threads():
    """batch * length just below 2^25 with more than 32 states: db and dc alone take 2^32 threads but for a few.  Every row holds the
    same tokens, so that one row in 64 bits says what all of them hold; da adds the rows up in FP64 and rounds once more."""
    batch, length, n = 20485, 1638, 33
    say(f"[ssm] batch={batch} length={length} d=1 n={n}")
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    one = dict(u=normal(1, length, 1).to(bf), dt=normal(1, length, 1).to(bf), a=-torch.rand(1, n, generator=g, device="cuda") - 0.1,
               b=normal(1, length, 1, n).to(bf), c=normal(1, length, 1, n).to(bf), d=normal(1), dt_bias=normal(1) - 2)
    dy = normal(1, length, 1).to(bf)
    k = {m: t.repeat(batch, *[1] * (t.dim() - 1)) if m in ("u", "dt", "b", "c") else t for m, t in one.items()}
    y, h, saved = ssm.ssm_scan_fwd(**k)
    got = ssm.ssm_scan_bwd(k["u"], k["dt"], k["a"], k["b"], k["c"], k["d"], None, k["dt_bias"], saved, dy.repeat(batch, 1, 1))
    torch.cuda.synchronize()
    got.update(y=y, h=h)
    ref = scan_ref(**one, dy=dy)
    tol = scan_tolerance(scan_ref(**one, dy=dy, absolute=True), ref, length, bf)
    for m, t in got.items():
        if m in ("da", "dd", "ddt_bias"):
            err, most = (t.double() - batch * ref[m]).abs(), batch * (tol[m] + U * ref[m].abs())
        else:
            assert (t == t[:1]).all(), m
            err, most = (t[:1].double() - ref[m]).abs(), tol[m]
        assert (err <= most).all(), (m, float(err.max()))


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_single_tokens_of_long_rows(dtype):
    """A token's slices of prompts whose rows lie 2^22 elements and more apart, as the same values one after the other."""
    batch, length, width, n = 3, 2049, 2048, 4
    say(f"[ssm] slices of long rows {dtype}")
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.randn(batch, length, width, generator=g, device="cuda").to(dtype)
    both = torch.randn(batch, length, 2 * n + 2040, generator=g, device="cuda").to(dtype)
    b, c = both[..., :n].unsqueeze(-2), both[..., n:2 * n].unsqueeze(-2)
    a, h = -torch.rand(width, n, generator=g, device="cuda"), torch.randn(batch, width, n, generator=g, device="cuda")
    for t in (0, 1000, length - 1):
        one, two = h.clone(), h.clone()
        assert u[:, t].stride(0) >= 1 << 22
        y = ssm.ssm_scan_step(one, u[:, t], u[:, t], a, b[:, t], c[:, t], z=u[:, t])
        x = u[:, t].contiguous()
        want = ssm.ssm_scan_step(two, x, x, a, b[:, t].contiguous(), c[:, t].contiguous(), z=x)
        assert torch.equal(y, want) and torch.equal(one, two) and not torch.equal(one, h)


@pytest.mark.parametrize("batch,length,d,n", [(32801, 1024, 1, 1), (1, 19, 1 << 21, 2)])
def test_many_tokens_and_wide_rows(batch, length, d, n):
    """More than 2^25 tokens, and the widest rows.  Every row holds the same tokens, and where it is wide the same channels over and over, so
    that few of them in 64 bits say what all hold; db and dc add the channels up."""
    say(f"[ssm] batch={batch} length={length} d={d} n={n}")
    g = torch.Generator(device="cuda").manual_seed(3)
    few = min(d, 32)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    one = dict(u=normal(1, length, few), dt=normal(1, length, few), a=-torch.rand(few, n, generator=g, device="cuda") - 0.1,
               b=normal(1, length, 1, n), c=normal(1, length, 1, n), d=normal(few), z=normal(1, length, few), dt_bias=normal(few) - 2)
    dy = normal(1, length, few)
    times = d // few
    k = {m: t.repeat(batch, 1, times) if m in ("u", "dt", "z") else t.repeat(batch, 1, 1, 1) if m in ("b", "c") else t.repeat(times, *[1] * (t.dim() - 1))
         for m, t in one.items()}
    y, h, saved = ssm.ssm_scan_fwd(**k)
    got = ssm.ssm_scan_bwd(*k.values(), saved, dy.repeat(batch, 1, times))
    torch.cuda.synchronize()
    got.update(y=y, h=h)
    ref = scan_ref(**one, dy=dy)
    tol = scan_tolerance(scan_ref(**one, dy=dy, absolute=True), ref, length, f32)
    for m, t in got.items():
        per, want, most = t, ref[m], tol[m]
        if m in ("y", "du", "ddt", "dz"):
            per = t.unflatten(2, (times, few))
            want, most = want[:, :, None], most[:, :, None]
        elif m == "h":
            per, want, most = t.unflatten(1, (times, few)), want[:, None], most[:, None]
        elif m in ("da", "dd", "ddt_bias"):                      # FP64 over the rows, rounded once more
            per, want, most = t.unflatten(0, (times, few)), want[None] * batch, (most + U * want.abs())[None] * batch
        else:                                                    # FP32 over 128 / g channels of a wave at a time, four waves, then workgroups one by one
            want, most = want * times, (most + (times + 64) * U * tol[m] / (20 * (2 * length + 6) * U)) * times
        assert ((per.double() - want).abs() <= most).all(), m
