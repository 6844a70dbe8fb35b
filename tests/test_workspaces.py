"""Workspaces and records that a caller hands over: what the bindings refuse (CPU)."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_sequence_amd", "libsamu_scan.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libsamu_scan.so not built")
bf, f32 = torch.bfloat16, torch.float32


def calls():
    """name -> a call that takes a workspace of the size it asks for, on host tensors."""
    from linear_recurrence_sequence_amd import lm, ssm
    x, g, s, v = torch.zeros(2, 5, 12, dtype=bf), torch.zeros(2, 5, 1, 4, dtype=bf), torch.zeros(12, 4), torch.zeros(12)
    saved = torch.zeros(ssm.lib().ssm_scan_saved_bytes(2, 5, 12, 4, 1), dtype=torch.uint8)
    t, e, h = torch.zeros(5, dtype=torch.int64), torch.zeros(9, 16, dtype=bf), torch.zeros(5, 16, dtype=bf)
    r, st = torch.zeros(5, 16), torch.zeros(5, 2)
    return dict(
        ssm_scan_fwd=lambda w: ssm.ssm_scan_fwd(x, x, s, g, g, workspace=w),
        ssm_scan_bwd=lambda w: ssm.ssm_scan_bwd(x, x, s, g, g, None, None, None, saved, x, workspace=w),
        causal_conv_bwd=lambda w: ssm.causal_conv_bwd(x, s, v, x, workspace=w),
        embed_bwd=lambda w: lm.embed_bwd(t, h, 9, workspace=w),
        linear_ce_fwd=lambda w: lm.linear_ce_fwd(h, e, t, workspace=w),
        block_norm_bwd=lambda w: lm.block_norm_bwd(r, h, None, None, None, torch.zeros(16), st, r, h, workspace=w),
    )


NAMES = ("ssm_scan_fwd", "ssm_scan_bwd", "causal_conv_bwd", "embed_bwd", "linear_ce_fwd", "block_norm_bwd")


@pytest.mark.parametrize("name", NAMES)
def test_a_workspace_that_is_not_dense(name):
    """One byte expanded counts as many, and a kernel would write behind it."""
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        calls()[name](torch.zeros(1, dtype=torch.uint8).expand(1 << 20))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        calls()[name](torch.zeros(2 << 20, dtype=torch.uint8)[::2])
    with pytest.raises(ValueError, match="device tensor"):
        calls()[name](torch.zeros(1 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("name", NAMES)
def test_a_workspace_of_another_device(name):
    with pytest.raises(ValueError, match="workspace is on meta, expected cpu"):
        calls()[name](torch.empty(1 << 20, dtype=torch.uint8, device="meta"))
