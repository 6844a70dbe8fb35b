"""What the language-model operators refuse, on the CPU: the binding before any
pointer reaches the library (host tensors are enough), and the C ABI before
anything is enqueued (made-up addresses, only where no GPU is visible)."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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
    from linear_recurrence_sequence_amd import lm
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lm_ops.h")).read(), flags=re.S)
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(lm_[a-z0-9_]*)\s*\(", text, flags=re.M))
    assert len(names) >= 4, names
    for n in names:
        assert hasattr(lm.lib(), n), f"{n} declared in lm_ops.h but not exported"


# ------------------------------------------------------------- block norms ---
def norm_args(**over):
    a = dict(x=torch.zeros(4, 24, dtype=f32), y=torch.zeros(4, 24, dtype=bf), gate=torch.zeros(4, 24, dtype=bf),
             w_post=torch.ones(24), scale=torch.ones(24), w_pre=torch.ones(24))
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,kw,msg", [
    (dict(x=torch.zeros(4, 24, dtype=torch.float16)), {}, "x has dtype"),
    (dict(y=torch.zeros(4, 23, dtype=bf)), {}, "y has shape"),
    (dict(gate=torch.zeros(4, 24)), {}, "gate has dtype"),
    (dict(gate=None), {}, "only with, a gate activation"),
    ({}, dict(gate_act="none"), "only with, a gate activation"),
    ({}, dict(gate_act="relu"), "gate_act must be one of"),
    (dict(scale=None), {}, "together or not at all"),
    (dict(w_post=None), {}, "together or not at all"),
    (dict(w_pre=None), {}, "w_pre is required"),
    (dict(w_pre=torch.ones(24, dtype=bf)), {}, "w_pre has dtype"),
    (dict(w_pre=torch.ones(48)[::2]), {}, "w_pre must be contiguous"),
    (dict(y=torch.zeros(4, 48, dtype=bf)[:, ::2]), {}, "y must have dense columns"),
    (dict(x=torch.zeros(2, 3, 2, 24)[:, :, 0][:, :2].transpose(0, 1).reshape(4, 24)), dict(r=torch.zeros(4, 24, dtype=bf)), "r has dtype"),
    ({}, dict(n=torch.zeros(4, 24)), "n has dtype"),
    ({}, dict(stats=torch.zeros(4, 1)), "stats has shape"),
    ({}, {}, "device tensor"),                                # well formed: only the device is wrong
])
def test_norm_binding_rejects(over, kw, msg):
    from linear_recurrence_sequence_amd import lm
    with pytest.raises(ValueError, match=msg):
        lm.block_norm_fwd(*norm_args(**over), **{"gate_act": "silu", **kw})


def test_norm_rows_at_several_distances_are_refused():
    from linear_recurrence_sequence_amd import lm
    x = torch.zeros(5, 4, 24)[:, :3]                          # rows at 24 within, 96 between
    a = [x, torch.zeros(5, 3, 24), None, None, None, torch.ones(24)]
    with pytest.raises(ValueError, match="rows at one distance"):
        lm._row_stride(x, "x")
    with pytest.raises(ValueError):
        lm.block_norm_fwd(*a)
    assert lm._row_stride(torch.zeros(5, 3, 48)[..., :24], "x") == 48
    assert lm._row_stride(torch.zeros(5, 1, 48)[..., :24], "x") == 48
    assert lm._row_stride(torch.zeros(1, 24).expand(5, 24), "x") == 0
    assert lm._row_stride(torch.zeros(0, 24), "x") == 24


def test_norm_bwd_binding_rejects():
    from linear_recurrence_sequence_amd import lm
    a = norm_args()
    ok = dict(stats=torch.zeros(4, 2), dr=torch.zeros(4, 24), dn=torch.zeros(4, 24, dtype=bf))
    for over, msg in ((dict(stats=torch.zeros(3, 2)), "stats has shape"), (dict(dr=torch.zeros(4, 24, dtype=bf)), "dr has dtype"),
                      (dict(dn=torch.zeros(4, 24)), "dn has dtype"), (dict(workspace=torch.zeros(8, dtype=torch.uint8)), "workspace holds"),
                      ({}, "device tensor")):
        kw = {**ok, **over}
        with pytest.raises(ValueError, match=msg):
            lm.block_norm_bwd(*a, kw.pop("stats"), kw.pop("dr"), kw.pop("dn"), gate_act="silu", **kw)


def P(n):
    return ctypes.c_void_p(n << 20)


def norm_fwd(**over):
    from linear_recurrence_sequence_amd import lm
    a = dict(rows=4, d=24, st=1, br=0, act=2, eps=1e-6, x=P(1), xs=24, y=P(2), ys=24, g=P(3), gs=24, w1=P(4), sc=P(5),
             w2=P(6), r=P(7), n=P(8), stats=P(9))
    a.update(over)
    return lm.lib().lm_block_norm_fwd(*a.values(), None)


@fake_pointers
@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), -2), (dict(d=0), -2), (dict(d=16385), -2), (dict(st=2), -2), (dict(act=3), -2), (dict(xs=-1), -2),
    (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2), (dict(g=None), -1), (dict(act=0), -2), (dict(sc=None), -1), (dict(x=None), -1),
    (dict(stats=None), -1), (dict(x=ctypes.c_void_p((1 << 20) + 2)), -3), (dict(y=ctypes.c_void_p((1 << 20) + 1)), -3),
    (dict(r=P(2)), -6), (dict(n=P(7)), -6), (dict(r=ctypes.c_void_p((1 << 20) + 4)), -6),
    (dict(xs=25, r=P(1)), -6), (dict(rows=0), 0),
])
def test_norm_abi_rejects(over, status):
    assert norm_fwd(**over) == status


@fake_pointers
def test_norm_bwd_abi_rejects():
    from linear_recurrence_sequence_amd import lm
    L = lm.lib()
    ok = dict(rows=4, d=24, st=1, br=0, act=2, x=P(1), xs=24, y=P(2), ys=24, g=P(3), gs=24, w1=P(4), sc=P(5), w2=P(6),
              stats=P(7), dr=P(8), drs=24, dn=P(9), dns=24, dx=P(10), dy=P(11), dg=P(12), dw1=P(13), ds=P(14), dw2=P(15),
              ws=P(16), wn=1 << 20)
    for over, status in ((dict(dg=None), -1), (dict(dw1=None), -1), (dict(dw2=None), -1), (dict(stats=None), -1), (dict(wn=8), -4),
                         (dict(dx=P(1)), -6), (dict(dy=P(9)), -6), (dict(dw1=P(14)), -6), (dict(ws=P(10)), -6), (dict(drs=-4), -2)):
        assert L.lm_block_norm_bwd(*{**ok, **over}.values(), None) == status, over
    assert L.lm_block_norm_bwd_workspace_bytes(-1, 24) == 0 and L.lm_block_norm_bwd_workspace_bytes(4, 0) == 0
    assert L.lm_block_norm_bwd_workspace_bytes(0, 24) > 0


# ---------------------------------------------------- linear cross entropy ---
def ce_args(**over):
    a = dict(h=torch.zeros(5, 24, dtype=bf), w=torch.zeros(40, 24, dtype=bf), target=torch.zeros(5, dtype=torch.int64))
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,kw,msg", [
    (dict(h=torch.zeros(5, 24)), {}, "h has dtype"),
    (dict(w=torch.zeros(40, 24)), {}, "w has dtype"),
    (dict(w=torch.zeros(40, 16, dtype=bf)), {}, "got shapes"),
    (dict(w=torch.zeros(24, 40, dtype=bf).t()), {}, "w must be contiguous"),
    (dict(h=torch.zeros(24, 5, dtype=bf).t()), {}, "h must have dense columns"),
    (dict(target=torch.zeros(5, dtype=torch.int32)), {}, "target has dtype"),
    (dict(target=torch.zeros(4, dtype=torch.int64)), {}, "target has shape"),
    (dict(h=torch.zeros(5, 20, dtype=bf), w=torch.zeros(40, 20, dtype=bf)), {}, "unsupported shape"),
    ({}, dict(loss=torch.zeros(5, dtype=bf)), "loss has dtype"),
    ({}, dict(lse=torch.zeros(6)), "lse has shape"),
    ({}, dict(workspace=torch.zeros(16, dtype=torch.uint8)), "workspace holds"),
    ({}, {}, "device tensor"),
])
def test_ce_binding_rejects(over, kw, msg):
    from linear_recurrence_sequence_amd import lm
    with pytest.raises(ValueError, match=msg):
        lm.linear_ce_fwd(*ce_args(**over), **kw)


def test_ce_bwd_binding_rejects():
    from linear_recurrence_sequence_amd import lm
    ok = dict(lse=torch.zeros(5), dloss=torch.zeros(5), dlse=torch.zeros(5))
    for over, msg in ((dict(lse=torch.zeros(4)), "lse has shape"), (dict(dloss=None), "dloss is required"),
                      (dict(dlse=torch.zeros(5, dtype=bf)), "dlse has dtype"), (dict(dh=torch.zeros(5, 24), dw=torch.zeros(40, 24, dtype=bf)), "dw has dtype"),
                      (dict(dw=torch.zeros(40, 23, dtype=bf)), "dw has shape"), (dict(grad_dtype=torch.float16), "output dtype"),
                      ({}, "device tensor")):
        kw = {**ok, **over}
        with pytest.raises(ValueError, match=msg):
            lm.linear_ce_bwd(*ce_args(), kw.pop("lse"), kw.pop("dloss"), kw.pop("dlse"), **kw)


@fake_pointers
def test_ce_abi_rejects():
    from linear_recurrence_sequence_amd import lm
    L = lm.lib()
    fwd = dict(n=5, d=24, v=40, cap=0.0, h=P(1), hs=24, w=P(2), t=P(3), loss=P(4), lse=P(5), ws=P(6), wn=1 << 20)
    for over, status in ((dict(n=-1), -2), (dict(d=20), -2), (dict(d=0), -2), (dict(d=65544), -2), (dict(v=0), -2), (dict(v=1 << 31), -2),
                         (dict(cap=-1.0), -2), (dict(cap=float("nan")), -2), (dict(cap=float("inf")), -2), (dict(hs=28), -2), (dict(hs=-24), -2),
                         (dict(hs=1 << 22), -2), (dict(h=None), -1), (dict(t=None), -1), (dict(h=ctypes.c_void_p((1 << 20) + 8)), -3),
                         (dict(w=ctypes.c_void_p((2 << 20) + 2)), -3), (dict(wn=16), -4), (dict(loss=P(3)), -6), (dict(lse=P(4)), -6),
                         (dict(n=0, h=None, t=None), 0)):
        assert L.lm_linear_ce_fwd(*{**fwd, **over}.values(), None) == status, over
    bwd = dict(n=5, d=24, v=40, cap=0.0, h=P(1), hs=24, w=P(2), t=P(3), lse=P(4), dl=P(5), dlse=P(6), dh=P(7), dw=P(8), gd=0, ws=P(9), wn=1 << 20)
    for over, status in ((dict(gd=2), -2), (dict(lse=None), -1), (dict(dl=None), -1), (dict(dh=None), -1), (dict(dw=None), -1), (dict(wn=16), -4),
                         (dict(dh=P(1)), -6), (dict(dw=P(2)), -6), (dict(ws=P(8)), -6), (dict(dw=ctypes.c_void_p((8 << 20) + 4)), -3),
                         (dict(n=0, dw=None), -1)):
        assert L.lm_linear_ce_bwd(*{**bwd, **over}.values(), None) == status, over
    assert L.lm_linear_ce_workspace_bytes(5, 20, 40, 1) == 0
    # pieces of the vocabulary: the backward's workspace does not grow with n v
    assert L.lm_linear_ce_workspace_bytes(8192, 2048, 128000, 1) < 8192 * 128000 // 2


# ------------------------------------------------------------------- AdamW ---
def adamw(**over):
    from linear_recurrence_sequence_amd import lm
    n = 300
    a = dict(params=[torch.zeros(n, dtype=bf)], grads=[torch.zeros(n, dtype=bf)], m=[torch.zeros(n)], v=[torch.zeros(n)])
    kw = dict(step=1, lr=1e-3, masters=[torch.zeros(n)])
    for k, x in over.items():
        (a if k in a else kw)[k] = x
    return lm.adamw_step(*a.values(), **kw)


@pytest.mark.parametrize("over,msg", [
    (dict(params=[torch.zeros(300, dtype=torch.float16)]), r"params\[0\] has dtype"),
    (dict(grads=[torch.zeros(299, dtype=bf)]), r"grads\[0\] must be"),
    (dict(grads=[]), "as long as each other"),
    (dict(m=[torch.zeros(300, dtype=bf)]), r"m\[0\] must be"),
    (dict(v=[torch.zeros(600)[::2]]), r"v\[0\] must be"),
    (dict(masters=[torch.zeros(300, dtype=bf)]), r"masters\[0\] must be"),
    (dict(masters=[]), "masters holds 0"),
    (dict(weight_decay=[0.1, 0.2]), "weight_decay holds 2"),
    (dict(m_scales=[torch.zeros(2)]), "together or not at all"),
    (dict(m_scales=[torch.zeros(2)], v_scales=[torch.zeros(2)]), r"m\[0\] must be"),    # FP32 states, 8-bit scales
    ({}, "device tensors"),
])
def test_adamw_binding_rejects(over, msg):
    with pytest.raises(ValueError, match=msg):
        adamw(**over)


def test_adamw_state_shapes():
    from linear_recurrence_sequence_amd import lm
    s = lm.adamw_state(torch.zeros(3, 200), 8)
    assert s["m"].dtype == torch.float8_e4m3fn and s["m"].shape == (3, 200) and s["v_scale"].shape == (3,)
    assert set(lm.adamw_state(torch.zeros(3))) == {"m", "v"}
    with pytest.raises(ValueError):
        lm.adamw_state(torch.zeros(3), 16)


@fake_pointers
def test_adamw_abi_rejects():
    from linear_recurrence_sequence_amd import lm

    def ptrs(*v):
        return None if v == (None,) else (ctypes.c_void_p * len(v))(*v)

    M = 1 << 20
    ok = dict(count=2, pd=0, gd=0, bits=8, p=ptrs(M, 2 * M), g=ptrs(3 * M, 4 * M), m=ptrs(5 * M, 6 * M), v=ptrs(7 * M, 8 * M),
              master=ptrs(9 * M, 10 * M), ms=ptrs(11 * M, 12 * M), vs=ptrs(13 * M, 14 * M), n=(ctypes.c_int64 * 2)(300, 5),
              decay=(ctypes.c_double * 2)(0, 0), lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, step=1)
    for over, status in ((dict(count=-1), -2), (dict(pd=2), -2), (dict(bits=16), -2), (dict(step=0), -2), (dict(b1=1.0), -2),
                         (dict(b2=-0.1), -2), (dict(eps=-1.0), -2), (dict(lr=float("nan")), -2), (dict(p=None), -1), (dict(ms=None), -1),
                         (dict(v=ptrs(7 * M, None)), -1), (dict(master=ptrs(9 * M, None)), -1), (dict(p=ptrs(M + 1, 2 * M)), -3),
                         (dict(ms=ptrs(11 * M + 2, 12 * M)), -3), (dict(p=ptrs(M, M)), -6),          # a tensor twice
                         (dict(g=ptrs(3 * M, 2 * M)), -6),                                           # a gradient that is a weight
                         (dict(m=ptrs(5 * M, 5 * M + 299)), -6), (dict(vs=ptrs(13 * M, 13 * M + 4)), -6),
                         (dict(n=(ctypes.c_int64 * 2)(-1, 5)), -2), (dict(count=0), 0),
                         (dict(n=(ctypes.c_int64 * 2)(0, 0)), 0)):
        assert lm.lib().lm_adamw_step(*{**ok, **over}.values(), None) == status, over
    # gradients may share memory (one tensor used twice as a gradient reads only)
    assert lm.lib().lm_adamw_step(*{**ok, "g": ptrs(3 * M, 3 * M), "p": ptrs(M, M)}.values(), None) == -6
