"""The embedding at vocabularies whose rows are more than one for each wave, up to the largest accepted one."""
import pytest
import torch

from linear_recurrence_sequence_amd import lm
from tests.helpers import say
from tests.ssm_ref import U, embed_ref, half_step

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("ot,gt", [(bf, bf), (f32, f32), (bf, f32)], ids=["bf16", "f32", "bf16_to_f32"])
@pytest.mark.parametrize("n,d,v", [(9000, 8, 65537), (3000, 33, 131073), (20000, 1, 700001)])
def test_rows_of_several_to_a_wave(ot, gt, n, d, v):
    """A wave takes a second row from 65536 rows on.  Sums of k values are off by less than k halves of a step of their sizes' sum, the
    scale takes one more, adding to what is there another; each result is rounded once."""
    say(f"[embed] wide {ot} {gt} n={n} d={d} v={v}")
    g = torch.Generator(device="cuda").manual_seed(n)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    r = torch.rand(n, generator=g, device="cuda")
    t = torch.where(r < 0.3, v - 1 - (t % 3), t)                   # the last rows have many
    t = torch.where(r > 0.95, torch.full_like(t, -1), t)
    dout = torch.randn(n, d, generator=g, device="cuda").to(ot)
    got, want, size = lm.embed_bwd(t, dout, v, scale=0.3, grad_dtype=gt), embed_ref(t, dout, v, 0.3), embed_ref(t, dout, v, 0.3, absolute=True)
    most = int(torch.bincount(t[t >= 0], minlength=v).max())
    assert ((got.double() - want).abs() <= (most + 2) * U * size + half_step(gt) * want.abs()).all()
    base = torch.randn(v, d, generator=g, device="cuda").to(gt)
    dw = lm.embed_bwd(t, dout, v, scale=0.3, dw=base.clone(), accumulate=True)
    total = base.double() + want
    assert ((dw.double() - total).abs() <= (most + 3) * U * (size + base.double().abs()) + half_step(gt) * total.abs()).all()


def test_the_largest_vocabulary():
    """The sort's launch is 1024 threads short of 2^32."""
    v = (2 ** 22 - 1) * 512
    say(f"[embed] v={v}")
    t = torch.tensor([v - 1, 0, v - 1, 12345678, -1, v, 2 ** 30], device="cuda")
    dout = torch.tensor([1.0, 2.0, 4.0, 8.0, 16.0, 32.0, 64.0], device="cuda")[:, None].to(bf)
    dw = lm.embed_bwd(t, dout, v)
    assert torch.equal(dw[t[[0, 1, 3, 6]], 0].float().cpu(), torch.tensor([5.0, 2.0, 8.0, 64.0]))
    assert sum(int(p.count_nonzero()) for p in dw.split(1 << 28)) == 4
    out = lm.embed_fwd(t, dw)
    assert torch.equal(out[[0, 1, 2, 3, 4, 6], 0].float().cpu(), torch.tensor([5.0, 2.0, 5.0, 8.0, 0.0, 64.0])) and out[5].isnan().all()


def test_the_most_tokens():
    """Seven rows of about 9.6 million tokens each: counts below 2^24, which FP32 adds up exactly in any order."""
    n, v = (1 << 26) - 64, 7
    say(f"[embed] n={n} v={v}")
    t = torch.randint(0, v, (n,), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    t[::1000] = -1
    counts = torch.bincount(t[t >= 0], minlength=v)
    assert int(counts.max()) < 1 << 24
    dout = torch.ones(1, 3, device="cuda").expand(n, 3)
    assert torch.equal(lm.embed_bwd(t, dout, v, grad_dtype=f32).double(), counts.double()[:, None].expand(v, 3))
    w = torch.arange(21, device="cuda", dtype=f32).view(v, 3) + 1
    out = lm.embed_fwd(t, w, out_dtype=bf)
    assert torch.equal(out[-70000:], torch.where((t[-70000:] >= 0)[:, None], w[t[-70000:].clamp_min(0)], 0).to(bf))
    assert torch.equal(out[:, 0].float(), torch.where(t >= 0, 3.0 * t + 1, 0.0))
