"""The embedding's largest vocabulary: what the sizes and the C ABI accept (CPU)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_sequence_amd", "libsamu_scan.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libsamu_scan.so not built")

# The sort has 1024 threads for each 512 rows of the vocabulary: below 2^32 threads up to 2^22 - 1 such workgroups.
MOST = (2 ** 22 - 1) * 512


def test_the_sort_stays_below_2_32_threads():
    from linear_recurrence_sequence_amd import lm
    size = lm.lib().lm_embed_bwd_workspace_bytes
    assert -(-MOST // 512) * 1024 < 2 ** 32 <= -(-(MOST + 1) // 512) * 1024
    assert size(5, 1, MOST) >= 4 * (MOST + 1) and size(5, 1, MOST + 1) == 0 and size(5, 1, 2 ** 31 - 256) == 0


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="made-up device addresses run only where no GPU is visible")
def test_the_calls_refuse_a_larger_vocabulary():
    from linear_recurrence_sequence_amd import lm
    p = [ctypes.c_void_p(n << 40) for n in (1, 2, 3, 4)]
    assert lm.lib().lm_embed_fwd(5, 1, MOST + 1, 0, 0, 1.0, p[0], p[1], p[2], None) == -2
    assert lm.lib().lm_embed_bwd(5, 1, MOST + 1, 0, 0, 1.0, p[0], p[1], 1, 0, p[2], p[3], 1 << 40, None) == -2
    assert b"2147483136" in lm.lib().scan_last_error()
