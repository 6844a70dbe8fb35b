"""Padded rows whose start flags reach into the padding: what each of the two operators of a block leaves, and how a program keeps the
states that single tokens go on from."""
import pytest
import torch

from linear_recurrence_sequence_amd import ssm
from tests.helpers import say

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_flags_in_padding(dtype):
    """As documented: a flag in the padding empties the scan's state and not the convolution's; without those flags both states are
    those of the row's last sequence alone: the convolution's to the bit, the scan's within 20 (2 * 50 + 6) halves of a step of the sizes added
    up, 1.3e-4, which are a few times the states'."""
    say(f"[ssm] flags in padding {dtype}")
    batch, length, d, n = 3, 60, 40, 16
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    x, dt, b, c = normal(batch, length, d), normal(batch, length, d), normal(batch, length, 1, n), normal(batch, length, 1, n)
    a, w = -torch.rand(d, n, generator=g, device="cuda") - 0.1, torch.randn(d, 4, generator=g, device="cuda")
    ends, starts = [33, 50, 60], [20, 0, 58]
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda")
    reset = torch.zeros(batch, length, dtype=torch.uint8, device="cuda")
    for i, (s, e) in enumerate(zip(starts, ends)):
        reset[i, s] = 1
        if e < length:
            reset[i, e] = 1                                      # as flags formed from the numbers of sequences and of the padding behind
    own = reset * (torch.arange(length, device="cuda") < lengths[:, None])
    _, h, _ = ssm.ssm_scan_fwd(x, dt, a, b, c, reset=reset, lengths=lengths)
    _, taps = ssm.causal_conv_fwd(x, w, reset=reset, lengths=lengths)
    _, kept, _ = ssm.ssm_scan_fwd(x, dt, a, b, c, reset=own, lengths=lengths)
    _, same = ssm.causal_conv_fwd(x, w, reset=own, lengths=lengths)
    assert torch.equal(taps, same) and not h[:2].any() and torch.equal(h[2], kept[2])
    for i, (s, e) in enumerate(zip(starts, ends)):
        k = slice(s, e)
        _, want, _ = ssm.ssm_scan_fwd(x[i:i + 1, k], dt[i:i + 1, k], a, b[i:i + 1, k], c[i:i + 1, k])
        _, last = ssm.causal_conv_fwd(x[i:i + 1, k], w)
        torch.testing.assert_close(kept[i:i + 1], want, rtol=1.3e-4, atol=1.3e-4)
        assert torch.equal(taps[i:i + 1], last)
