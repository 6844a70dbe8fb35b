"""What the selective scan, the convolution and the embedding refuse, on the CPU: the binding before any pointer reaches the
library (host tensors are enough), and the C ABI before anything is enqueued (made-up addresses, only where no GPU is visible)."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_recurrence_sequence_amd", "csrc")
LIB = os.path.join(ROOT, "linear_recurrence_sequence_amd", "libsamu_scan.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libsamu_scan.so not built")
bf, f32 = torch.bfloat16, torch.float32


def _gpu_visible():
    return torch.cuda.device_count() > 0    # counts devices without initializing them


fake_pointers = pytest.mark.skipif(_gpu_visible(), reason="made-up device addresses run only where no GPU is visible "
                                                          "(see test_rejections_in_a_gpu_free_child)")


@pytest.mark.skipif(not _gpu_visible(), reason="the rejection tests run in this process")
def test_rejections_in_a_gpu_free_child():
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="", CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", __file__],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


def test_every_declared_symbol_is_exported():
    from linear_recurrence_sequence_amd import ssm
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ssm_ops.h")).read(), flags=re.S)
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(ssm_[a-z0-9_]*)\s*\(", text, flags=re.M))
    assert len(names) == 9, names
    for n in names:
        assert hasattr(ssm.lib(), n), f"{n} declared in ssm_ops.h but not exported"


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_the_plan(tmp_path):
    exe = str(tmp_path / "ssm_plan_harness")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", f"-I{CSRC}",
                        os.path.join(ROOT, "tests", "sanitize", "ssm_plan_harness.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe, "20000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all walked" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


# ------------------------------------------------------------------- scan ---
def scan_args(lead=(2, 5), **over):
    a = dict(u=torch.zeros(*lead, 12, dtype=bf), dt=torch.zeros(*lead, 12, dtype=bf), a=torch.zeros(12, 4), b=torch.zeros(*lead, 2, 4, dtype=bf),
             c=torch.zeros(*lead, 2, 4, dtype=bf), d=torch.zeros(12), z=torch.zeros(*lead, 12, dtype=bf), dt_bias=torch.zeros(12))
    a.update(over)
    return list(a.values())


BAD_SCAN = [
    (dict(u=torch.zeros(2, 5, 12, dtype=torch.float16)), "u has dtype"),
    (dict(u=torch.zeros(5, 12, 3, 2, dtype=bf)), "u must be"),
    (dict(dt=torch.zeros(2, 5, 12)), "dt has dtype"),
    (dict(dt=torch.zeros(2, 4, 12, dtype=bf)), "dt has shape"),
    (dict(a=torch.zeros(12, 4, dtype=bf)), "a has dtype"),
    (dict(a=torch.zeros(11, 4)), "a must be"),
    (dict(a=torch.zeros(12, 65)), "a must be"),
    (dict(a=torch.zeros(4, 12).t()), "a must be contiguous"),
    (dict(b=torch.zeros(2, 5, 5, 4, dtype=bf)), "b must be"),
    (dict(b=torch.zeros(2, 5, 4, dtype=bf)), "b must be"),
    (dict(c=torch.zeros(2, 5, 1, 4, dtype=bf)), "c has shape"),
    (dict(b=torch.zeros(2, 5, 4, 2, dtype=bf).transpose(2, 3)), "b must have dense rows"),
    (dict(d=torch.zeros(12, dtype=bf)), "d has dtype"),
    (dict(dt_bias=torch.zeros(24)[::2]), "dt_bias must be contiguous"),
    (dict(z=torch.zeros(2, 5, 24, dtype=bf)[..., ::2]), "z must have dense columns"),
    ({}, "device tensor"),
]


@pytest.mark.parametrize("over,msg", BAD_SCAN)
def test_scan_binding_rejects(over, msg):
    from linear_recurrence_sequence_amd import ssm
    with pytest.raises(ValueError, match=msg):
        ssm.ssm_scan_fwd(*scan_args(**over))


@pytest.mark.parametrize("kw,msg", [
    (dict(h0=torch.zeros(2, 4, 12)), "h0 has shape"), (dict(h0=torch.zeros(2, 12, 4, dtype=bf)), "h0 has dtype"),
    (dict(reset=torch.zeros(2, 5)), "reset has dtype"), (dict(reset=torch.zeros(2, 4, dtype=torch.uint8)), "reset has shape"),
    (dict(reset=torch.zeros(5, 2, dtype=torch.uint8).t()), "reset must be contiguous"),
    (dict(lengths=torch.zeros(2, dtype=torch.int64)), "lengths has dtype"), (dict(lengths=torch.zeros(3, dtype=torch.int32)), "lengths has shape"),
    (dict(y=torch.zeros(2, 5, 12)), "y has dtype"), (dict(h_final=torch.zeros(2, 12, 5)), "h_final has shape"),
    (dict(workspace=torch.zeros(16, dtype=torch.uint8)), "workspace holds"),
])
def test_scan_options_rejected(kw, msg):
    from linear_recurrence_sequence_amd import ssm
    with pytest.raises(ValueError, match=msg):
        ssm.ssm_scan_fwd(*scan_args(), **kw)


def test_scan_bwd_and_step_reject():
    from linear_recurrence_sequence_amd import ssm
    saved = torch.zeros(ssm.lib().ssm_scan_saved_bytes(2, 5, 12, 4, 2), dtype=torch.uint8)
    ok = dict(saved=saved, dy=torch.zeros(2, 5, 12, dtype=bf), dh_final=torch.zeros(2, 12, 4))
    for over, msg in ((dict(saved=saved[:-1]), "saved has shape"), (dict(dy=None), "dy is required"), (dict(dy=torch.zeros(2, 5, 12)), "dy has dtype"),
                      (dict(dh_final=torch.zeros(2, 12, 3)), "dh_final has shape"), ({}, "device tensor")):
        kw = {**ok, **over}
        with pytest.raises(ValueError, match=msg):
            ssm.ssm_scan_bwd(*scan_args(), kw.pop("saved"), kw.pop("dy"), kw.pop("dh_final"))
    h = torch.zeros(2, 12, 4)
    for a, state, msg in ((scan_args(lead=(2,)), h[:, :, :3], "h has shape"), (scan_args(lead=(2,)), h.to(bf), "h has dtype"), (scan_args(), h, "u must be"),
                          (scan_args(lead=(2,)), torch.zeros(2, 4, 12).transpose(1, 2), "h must be contiguous"), (scan_args(lead=(2,)), h, "device tensor")):
        with pytest.raises(ValueError, match=msg):
            ssm.ssm_scan_step(state, *a)


def P(n):
    return ctypes.c_void_p(n << 20)


@fake_pointers
def test_scan_abi_rejects():
    from linear_recurrence_sequence_amd import ssm
    L = ssm.lib()
    fwd = dict(batch=2, length=5, d=12, n=4, groups=2, dtype=0, sp=1, u=P(1), us=12, dt=P(2), dts=12, a=P(3), b=P(4), bs=8, c=P(5), cs=8, skip=P(6),
               z=P(7), zs=12, bias=P(8), h0=P(9), reset=P(10), lengths=P(11), y=P(12), h=P(13), saved=P(14), ws=P(15), wn=1 << 20)
    for over, status in ((dict(batch=-1), -2), (dict(length=-1), -2), (dict(d=0), -2), (dict(d=13), -2), (dict(d=1 << 22), -2), (dict(n=0), -2),
                         (dict(n=65), -2), (dict(groups=0), -2), (dict(groups=5), -2), (dict(dtype=2), -2), (dict(us=-1), -2), (dict(bs=1 << 22), -2),
                         (dict(batch=1 << 16, length=1 << 15), -2), (dict(u=None), -1), (dict(a=None), -1), (dict(c=None), -1), (dict(y=None), -1),
                         (dict(h=None), -1), (dict(ws=None), -1), (dict(u=ctypes.c_void_p((1 << 20) + 1)), -3), (dict(a=ctypes.c_void_p((3 << 20) + 2)), -3),
                         (dict(saved=ctypes.c_void_p((14 << 20) + 4)), -3), (dict(wn=8), -4), (dict(y=P(1)), -6), (dict(h=P(9)), -6), (dict(y=P(7)), -6),
                         (dict(saved=P(13)), -6), (dict(ws=P(12)), -6), (dict(batch=0, u=None), 0)):
        assert L.ssm_scan_fwd(*{**fwd, **over}.values(), None) == status, over
    bwd = dict(batch=2, length=5, d=12, n=4, groups=2, dtype=0, sp=1, u=P(1), us=12, dt=P(2), dts=12, a=P(3), b=P(4), bs=8, c=P(5), cs=8, skip=P(6),
               z=P(7), zs=12, bias=P(8), reset=P(10), lengths=P(11), saved=P(12), dy=P(13), dys=12, dh=P(14), du=P(15), ddt=P(16), da=P(17), db=P(18),
               dc=P(19), ds=P(20), dz=P(21), dbias=P(22), dh0=P(23), ws=P(24), wn=1 << 20)
    for over, status in ((dict(n=65), -2), (dict(dys=-4), -2), (dict(saved=None), -1), (dict(dy=None), -1), (dict(du=None), -1), (dict(da=None), -1),
                         (dict(dz=None), -1), (dict(wn=8), -4), (dict(du=P(1)), -6), (dict(db=P(19)), -6), (dict(dh0=P(14)), -6), (dict(ws=P(17)), -6),
                         (dict(da=ctypes.c_void_p((17 << 20) + 2)), -3)):
        assert L.ssm_scan_bwd(*{**bwd, **over}.values(), None) == status, over
    step = dict(batch=2, d=12, n=4, groups=2, dtype=0, sp=1, h=P(1), u=P(2), us=12, dt=P(3), dts=12, a=P(4), b=P(5), bs=8, c=P(6), cs=8, skip=P(7), z=P(8),
                zs=12, bias=P(9), y=P(10))
    for over, status in ((dict(d=13), -2), (dict(h=None), -1), (dict(y=None), -1), (dict(h=P(2)), -6), (dict(y=P(1)), -6),
                         (dict(h=ctypes.c_void_p((1 << 20) + 2)), -3), (dict(batch=0), 0)):
        assert L.ssm_scan_step(*{**step, **over}.values(), None) == status, over
    assert L.ssm_scan_workspace_bytes(2, 5, 12, 65, 1, 0) == 0 and L.ssm_scan_saved_bytes(2, 5, 13, 4, 2) == 0


# ------------------------------------------------------------ convolution ---
@pytest.mark.parametrize("over,kw,msg", [
    (dict(x=torch.zeros(2, 5, 12, dtype=torch.float16)), {}, "x has dtype"),
    (dict(x=torch.zeros(5, 12)), {}, "x must be"),
    (dict(w=torch.zeros(12, 5)), {}, "w must be"),
    (dict(w=torch.zeros(12, 1)), {}, "w must be"),
    (dict(w=torch.zeros(11, 4)), {}, "w must be"),
    (dict(w=torch.zeros(12, 4, dtype=bf)), {}, "w has dtype"),
    (dict(w=torch.zeros(4, 12).t()), {}, "w must be contiguous"),
    (dict(bias=torch.zeros(11)), {}, "bias has shape"),
    ({}, dict(act="relu"), "act must be one of"),
    ({}, dict(state=torch.zeros(2, 3, 12)), "state has dtype"),
    ({}, dict(state=torch.zeros(2, 4, 12, dtype=bf)), "state has shape"),
    ({}, dict(reset=torch.zeros(2, 5)), "reset has dtype"),
    ({}, dict(lengths=torch.zeros(2)), "lengths has dtype"),
    ({}, dict(state_out=torch.zeros(2, 3, 11, dtype=bf)), "state_out has shape"),
    ({}, {}, "device tensor"),
])
def test_conv_binding_rejects(over, kw, msg):
    from linear_recurrence_sequence_amd import ssm
    a = dict(x=torch.zeros(2, 5, 12, dtype=bf), w=torch.zeros(12, 4), bias=torch.zeros(12))
    a.update(over)
    with pytest.raises(ValueError, match=msg):
        ssm.causal_conv_fwd(*a.values(), **kw)


def test_conv_bwd_and_step_reject():
    from linear_recurrence_sequence_amd import ssm
    x, w, b, dy = torch.zeros(2, 5, 12, dtype=bf), torch.zeros(12, 4), torch.zeros(12), torch.zeros(2, 5, 12, dtype=bf)
    for args, kw, msg in (((x, w, b, None), {}, "dy is required"), ((x, w, b, dy.float()), {}, "dy has dtype"),
                          ((x, w, b, dy, torch.zeros(2, 2, 12, dtype=bf)), {}, "dstate_out has shape"),
                          ((x, w, b, dy), dict(workspace=torch.zeros(8, dtype=torch.uint8)), "workspace holds"), ((x, w, b, dy), {}, "device tensor")):
        with pytest.raises(ValueError, match=msg):
            ssm.causal_conv_bwd(*args, **kw)
    for args, msg in (((x, w, b, torch.zeros(2, 3, 12, dtype=bf)), "x must be"), ((x[:, 0], w, b, None), "state is required"),
                      ((x[:, 0], w, b, torch.zeros(2, 3, 12)), "state has dtype"), ((x[:, 0], w, b, torch.zeros(2, 3, 12, dtype=bf)), "device tensor")):
        with pytest.raises(ValueError, match=msg):
            ssm.causal_conv_step(*args)


@fake_pointers
def test_conv_abi_rejects():
    from linear_recurrence_sequence_amd import ssm
    L = ssm.lib()
    fwd = dict(batch=2, length=5, d=12, width=4, dtype=0, act=1, x=P(1), xs=12, w=P(2), bias=P(3), state=P(4), reset=P(5), lengths=P(6), y=P(7), out=P(8))
    for over, status in ((dict(d=0), -2), (dict(width=1), -2), (dict(width=5), -2), (dict(dtype=3), -2), (dict(act=2), -2), (dict(xs=-1), -2),
                         (dict(batch=1 << 16, length=1 << 15), -2), (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(y=P(1)), -6),
                         (dict(out=P(4)), -6), (dict(out=P(7)), -6), (dict(x=ctypes.c_void_p((1 << 20) + 1)), -3), (dict(batch=0), 0)):
        assert L.ssm_conv_fwd(*{**fwd, **over}.values(), None) == status, over
    bwd = dict(batch=2, length=5, d=12, width=4, dtype=0, act=1, x=P(1), xs=12, w=P(2), bias=P(3), state=P(4), reset=P(5), lengths=P(6), dy=P(7), dys=12,
               do=P(8), dx=P(9), dw=P(10), db=P(11), ds=P(12), ws=P(13), wn=1 << 20)
    for over, status in ((dict(width=5), -2), (dict(dy=None), -1), (dict(dx=None), -1), (dict(dw=None), -1), (dict(wn=8), -4), (dict(dx=P(7)), -6),
                         (dict(ds=P(8)), -6), (dict(ws=P(10)), -6)):
        assert L.ssm_conv_bwd(*{**bwd, **over}.values(), None) == status, over
    step = dict(batch=2, d=12, width=4, dtype=0, act=1, x=P(1), xs=12, w=P(2), bias=P(3), state=P(4), y=P(5))
    for over, status in ((dict(act=-1), -2), (dict(state=None), -1), (dict(state=P(1)), -6), (dict(y=P(4)), -6), (dict(batch=0), 0)):
        assert L.ssm_conv_step(*{**step, **over}.values(), None) == status, over


# -------------------------------------------------------------- embedding ---
def test_embed_binding_rejects():
    from linear_recurrence_sequence_amd import lm
    t, w, g = torch.zeros(5, dtype=torch.int64), torch.zeros(9, 12, dtype=bf), torch.zeros(5, 12, dtype=bf)
    for args, kw, msg in (((t.int(), w), {}, "tokens has dtype"), ((t, w.half()), {}, "w has dtype"), ((t, w[0]), {}, "w must be"),
                          ((t, w.t()), {}, "w must be contiguous"), ((t.repeat(2)[::2], w), {}, "tokens must be contiguous"),
                          ((t, w), dict(out_dtype=torch.float16), "output dtype"), ((t, w), dict(out=torch.zeros(5, 11, dtype=bf)), "out has shape"),
                          ((t, w), {}, "device tensor")):
        with pytest.raises(ValueError, match=msg):
            lm.embed_fwd(*args, **kw)
    for args, kw, msg in (((t.int(), g, 9), {}, "tokens has dtype"), ((t, g.half(), 9), {}, "dout has dtype"), ((t[:4], g, 9), {}, "dout must be"),
                          ((t, g, 0), {}, "v must be"), ((t, g, 9), dict(accumulate=True), "needs a dw"), ((t, g, 9), dict(grad_dtype=torch.float16), "output dtype"),
                          ((t, g, 9), dict(dw=torch.zeros(8, 12)), "dw has shape"), ((t, g.t().contiguous().t(), 9), {}, "dout must have dense columns"),
                          ((t, g, 9), dict(workspace=torch.zeros(8, dtype=torch.uint8)), "workspace holds"), ((t, g, 9), {}, "device tensor")):
        with pytest.raises(ValueError, match=msg):
            lm.embed_bwd(*args, **kw)


@fake_pointers
def test_embed_abi_rejects():
    from linear_recurrence_sequence_amd import lm
    L = lm.lib()
    fwd = dict(n=5, d=12, v=9, wt=0, ot=1, scale=1.0, t=P(1), w=P(2), out=P(3))
    for over, status in ((dict(n=-1), -2), (dict(n=1 << 26), -2), (dict(d=0), -2), (dict(d=(1 << 23) + 1), -2), (dict(v=0), -2), (dict(v=1 << 31), -2), (dict(wt=2), -2),
                         (dict(ot=-1), -2), (dict(scale=float("inf")), -2), (dict(t=None), -1), (dict(out=None), -1), (dict(t=ctypes.c_void_p((1 << 20) + 4)), -3),
                         (dict(out=P(2)), -6), (dict(n=0, t=None), 0)):
        assert L.lm_embed_fwd(*{**fwd, **over}.values(), None) == status, over
    bwd = dict(n=5, d=12, v=9, ot=0, gt=1, scale=1.0, t=P(1), g=P(2), gs=12, add=0, dw=P(3), ws=P(4), wn=1 << 20)
    for over, status in ((dict(v=0), -2), (dict(gt=2), -2), (dict(gs=-1), -2), (dict(scale=float("nan")), -2), (dict(g=None), -1), (dict(dw=None), -1),
                         (dict(wn=16), -4), (dict(dw=P(2)), -6), (dict(ws=P(3)), -6), (dict(dw=ctypes.c_void_p((3 << 20) + 2)), -3),
                         (dict(n=0, t=None, g=None, add=1), 0)):
        assert L.lm_embed_bwd(*{**bwd, **over}.values(), None) == status, over
    assert L.lm_embed_bwd_workspace_bytes(5, 0, 9) == 0 and L.lm_embed_bwd_workspace_bytes(0, 12, 9) > 0
