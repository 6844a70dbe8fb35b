"""The linear cross entropy's plan on the CPU: the chunks, tiles and ranges that its launches take, over sizes across the
accepted range (built with the host compiler under both sanitizers)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_recurrence_sequence_amd", "csrc")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


def test_every_chunk_writes_what_is_summed(tmp_path):
    exe = str(tmp_path / "ce_plan_harness")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", f"-I{CSRC}",
                        os.path.join(ROOT, "tests", "sanitize", "ce_plan_harness.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe, "6000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "all walked" in r.stdout


def test_sizes_beyond_the_limits_are_refused():
    """The size query says 0, and a call fails, before anything is launched."""
    from linear_recurrence_sequence_amd import lm
    size = lm.lib().lm_linear_ce_workspace_bytes
    for n, d, v in (((1 << 26) - 16, 8, 5), (1 << 22, 4088, 300), (1, 8, (1 << 31) - 514), ((1 << 34) // 65536 - 1, 65536, 9)):
        assert size(n, d, v, 0) > 0 and size(n, d, v, 1) > 0, (n, d, v)
    for n, d, v in (((1 << 26) - 15, 8, 5), (1 << 22, 4096, 300), (1, 8, (1 << 31) - 513), (1 << 25, 512, 5), (1 << 24, 8, (1 << 31) - 514)):
        assert size(n, d, v, 0) == 0 and size(n, d, v, 1) == 0, (n, d, v)
