"""Launches of the selective scan at the widest sizes that it accepts (CPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_recurrence_sequence_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_the_last_launch(tmp_path):
    exe = str(tmp_path / "ssm_launch_harness")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", f"-I{CSRC}",
                        os.path.join(ROOT, "tests", "sanitize", "ssm_launch_harness.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all covered" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
