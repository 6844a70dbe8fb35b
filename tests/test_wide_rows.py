"""Widths that a C int does not hold: refused by the bindings before they are cut to 32 bits (CPU, tensors without memory)."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_sequence_amd", "libsamu_scan.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libsamu_scan.so not built")
bf, f32 = torch.bfloat16, torch.float32


def meta(*shape, dtype=bf):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("d", [(1 << 32) + 8, 1 << 31, (1 << 24) + 1])
def test_refused(d):
    """2^32 + 8 columns would else be taken for 8."""
    from linear_recurrence_sequence_amd import lm, ssm
    x, a, b, v = meta(1, 2, d), meta(d, 4, dtype=f32), meta(1, 2, 1, 4), meta(d, dtype=f32)
    t = torch.empty(2, dtype=torch.int64, device="meta")
    saved = torch.empty(256, dtype=torch.uint8, device="meta")
    calls = [lambda: ssm.ssm_scan_fwd(x, x, a, b, b), lambda: ssm.ssm_scan_bwd(x, x, a, b, b, None, None, None, saved, x),
             lambda: ssm.ssm_scan_step(meta(1, d, 4, dtype=f32), x[:, 0], x[:, 0], a, b[:, 0], b[:, 0]),
             lambda: ssm.causal_conv_fwd(x, a, v), lambda: ssm.causal_conv_bwd(x, a, v, x), lambda: ssm.causal_conv_step(x[:, 0], a, v, meta(1, 3, d)),
             lambda: lm.embed_fwd(t, meta(9, d)), lambda: lm.embed_bwd(t, x[0], 9)]
    for f in calls:
        with pytest.raises(ValueError, match="up to"):
            f()
