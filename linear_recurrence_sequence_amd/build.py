"""Build libsamu_scan.so (gfx950) in-tree with hipcc, and _lm_bind.so with g++.

    python -m linear_recurrence_sequence_amd.build [-v]

Every HIP source under csrc/ is compiled for gfx950 only, with packed FP32
instructions disabled, then linked into one shared library next to this file.
The binding module links to it and to torch, and is found by its place.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libsamu_scan.so")
BIND = os.path.join(HERE, "_lm_bind.so")
ARCH = "gfx950"

SOURCES = ["capi.cpp", "prefix.hip", "samu_fwd.hip", "samu_bwd.hip", "samu_decode.hip", "rglru.hip", "baseline.hip", "gate_proj.hip", "noalloc.hip",
           "lm_capi.cpp", "lm_norm.hip", "lm_adamw.hip", "lm_ce.hip", "lm_embed.hip", "ssm_capi.cpp", "ssm_fwd.hip", "ssm_bwd.hip", "ssm_conv.hip"]

CXXFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _hipcc():
    h = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(h):
        raise RuntimeError("hipcc not found (ROCm is required to build the HIP library)")
    return h


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_hipcc(), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj] + CXXFLAGS
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature and says so; that is harmless
    noise = "'-packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if verbose and err.strip():
        print(err, flush=True)
    return obj


def _bind(verbose):
    """The Python module of the operators' usual calls (host code)."""
    import sysconfig

    import torch
    at = os.path.dirname(torch.__file__)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", *[os.path.join(CSRC, f) for f in ("lm_bind.cpp", "ssm_bind.cpp")], "-o", BIND + ".tmp",
           f"-I{INCLUDE}", f"-I{at}/include", "-I" + sysconfig.get_paths()["include"],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-L{HERE}", "-l:" + os.path.basename(LIB), f"-L{at}/lib", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on the binding module:\n{r.stderr}")
    os.replace(BIND + ".tmp", BIND)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES), max(1, min(8, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    _bind(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
