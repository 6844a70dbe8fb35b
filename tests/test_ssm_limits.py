"""Sizes and strides that the selective scan accepts, by call (CPU)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_sequence_amd", "libsamu_scan.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libsamu_scan.so not built")
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="made-up device addresses run only where no GPU is visible")


def P(n):
    return ctypes.c_void_p(n << 40)


@no_gpu
def test_single_tokens_take_wide_row_strides():
    """A token's slice of a batch of prompts: rows lie length * d apart.  A state at u's address is refused behind the strides' check,
    so that nothing is launched."""
    from linear_recurrence_sequence_amd import ssm
    step = dict(batch=2, d=12, n=4, groups=2, dtype=0, sp=1, h=P(1), u=P(2), us=12, dt=P(3), dts=12, a=P(4), b=P(5), bs=8, c=P(6), cs=8, skip=P(7),
                z=P(8), zs=12, bias=P(9), y=P(10))
    f = ssm.lib().ssm_scan_step
    for name in ("us", "dts", "bs", "cs", "zs"):
        for stride, status in ((1 << 22, -6), (1 << 33, -6), ((1 << 40) + 1, -2), (-1, -2)):
            assert f(*{**step, name: stride, "h": P(4)}.values(), None) == status, (name, stride)


def test_documented_sizes_are_accepted():
    """batch * length below 2^31, d up to 2^21, and launches of fewer than 2^24 waves forward: nothing else bounds the sizes."""
    from linear_recurrence_sequence_amd import ssm
    size, saved = ssm.lib().ssm_scan_workspace_bytes, ssm.lib().ssm_scan_saved_bytes
    for batch, length, d, n, groups, ok in ((1, 1 << 25, 1, 1, 1, True), (1, (1 << 31) - 257, 1, 64, 1, True), (1, 1 << 20, 64, 64, 64, True),
                                            (1, 4, 1 << 21, 64, 1, True), (1, 4, (1 << 21) + 1, 1, 1, False), (64, 4, (1 << 21) - 8, 64, 1, True),
                                            (65, 4, 1 << 21, 64, 1, False), ((1 << 24) - 1, 1, 1, 1, 1, True), (1 << 24, 1, 1, 1, 1, False),
                                            (1 << 16, 1 << 15, 1, 1, 1, False)):
        case = batch, length, d, n, groups
        assert bool(size(*case, 0)) is ok and bool(size(*case, 1)) is ok and bool(saved(*case)) is ok, case
