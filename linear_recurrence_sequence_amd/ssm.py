"""The selective state space mixer: thin Python binding of the C ABI in
include/ssm_ops.h.

The scan with its gate, forward, backward and for single tokens, and the short
causal convolution in front of it.  Argument checks and marshalling only: every
step runs in the HIP kernels of libsamu_scan.so, on the current stream or the
one given.  The differentiable forms are in autograd.py.

With a stream given a call runs as if that stream were the current one: its
outputs and workspace are allocated there.  Tensors lie on the current device,
or the stream's.  The usual calls, right and with outputs of their own, go through
_lm_bind (csrc/ssm_bind.cpp); every other one is checked, and where it is wrong refused, here.

Rows of activations may lie apart (views of a wider projection).  In all calls
over several tokens, reset [batch, length] (uint8 or bool) marks tokens that
start a sequence, and lengths [batch] (int32) says where a row's padding begins: its
outputs and gradients are zero, and the state behind a row is the one after its
last token.  Of the scan it is zero if a token of the padding is marked, an empty sequence
starting there, while the convolution looks at no marks in the padding: where single tokens go
on from both states, clear those marks first, reset & (arange(length) < lengths[:, None]).
"""
import ctypes

import torch

from . import scan
from .lm import _dense, _native, _p, _row_stride, _same_device, _written
from .scan import _check, _code, _nbytes, _stream, _want, _want_bytes

_BF16, _F32 = torch.bfloat16, torch.float32
_DTYPES = (_BF16, _F32)
_FLAGS = (torch.uint8, torch.bool)
ACTS = {"none": 0, "silu": 1}
MAX_STATE, MAX_WIDTH = 64, 4
MAX_SCAN_D, MAX_CONV_D = 1 << 21, 1 << 24

_lib = None


def lib():
    """The loaded library with the argument types of ssm_ops.h."""
    global _lib
    if _lib is not None:
        return _lib
    L = scan.lib()
    i, i64, sz, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    row = [vp, i64]
    L.ssm_scan_saved_bytes.argtypes = [i64, i64, i, i, i]
    L.ssm_scan_saved_bytes.restype = sz
    L.ssm_scan_workspace_bytes.argtypes = [i64, i64, i, i, i, i]
    L.ssm_scan_workspace_bytes.restype = sz
    L.ssm_scan_fwd.argtypes = [i64, i64, i, i, i, i, i] + row * 2 + [vp] + row * 2 + [vp] + row + [vp] * 7 + [vp, sz, vp]
    L.ssm_scan_bwd.argtypes = [i64, i64, i, i, i, i, i] + row * 2 + [vp] + row * 2 + [vp] + row + [vp] * 4 + row + [vp] * 10 + [vp, sz, vp]
    L.ssm_scan_step.argtypes = [i64, i, i, i, i, i, vp] + row * 2 + [vp] + row * 2 + [vp] + row + [vp, vp, vp]
    L.ssm_conv_fwd.argtypes = [i64, i64, i, i, i, i] + row + [vp] * 8
    L.ssm_conv_bwd_workspace_bytes.argtypes = [i64, i64, i, i]
    L.ssm_conv_bwd_workspace_bytes.restype = sz
    L.ssm_conv_bwd.argtypes = [i64, i64, i, i, i, i] + row + [vp] * 5 + row + [vp] * 5 + [vp, sz, vp]
    L.ssm_conv_step.argtypes = [i64, i, i, i, i] + row + [vp] * 5
    for n in ("ssm_scan_fwd", "ssm_scan_bwd", "ssm_scan_step", "ssm_conv_fwd", "ssm_conv_bwd", "ssm_conv_step"):
        getattr(L, n).restype = i
    _lib = L
    return L


def _vector(t, name, n, optional=True):
    _want(t, name, _F32, (n,), optional=optional)
    _dense(t, name)


def _group_stride(t, name):
    """Row stride of b or c [..., groups, n], whose rows' groups * n values are dense."""
    g, n = t.shape[-2:]
    if (n > 1 and t.stride(-1) != 1) or (g > 1 and t.stride(-2) != n):
        raise ValueError(f"{name} must have dense rows (groups x n values one after the other)")
    flat = t.as_strided((*t.shape[:-2], g * n), (*t.stride()[:-2], 1))
    return _row_stride(flat, name)


def _out(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _want(t, name, dtype, shape)
    _dense(t, name)
    return t


def _sequence_args(lead, reset, lengths):
    _want(reset, "reset", _FLAGS, lead, optional=True)
    _want(lengths, "lengths", torch.int32, lead[:1], optional=True)
    _dense(reset, "reset")
    _dense(lengths, "lengths")


def _scan_args(u, dt, a, b, c, d, z, dt_bias, dims):
    """Checks what all calls of the scan share; returns (d, n, groups, row strides of u, dt, b, c, z)."""
    _want(u, "u", _DTYPES)
    if u.dim() != dims or not 1 <= u.shape[-1] <= MAX_SCAN_D:
        raise ValueError(f"u must be [batch{', length' if dims == 3 else ''}, d] with d from 1 up to {MAX_SCAN_D}, got shape {tuple(u.shape)}")
    lead, width = u.shape[:-1], u.shape[-1]
    _want(dt, "dt", u.dtype, u.shape)
    _want(z, "z", u.dtype, u.shape, optional=True)
    _want(a, "a", _F32)
    if a.dim() != 2 or a.shape[0] != width or not 1 <= a.shape[1] <= MAX_STATE:
        raise ValueError(f"a must be [d, n] with n in 1..{MAX_STATE}, got shape {tuple(a.shape)}")
    n = a.shape[1]
    _dense(a, "a")
    _want(b, "b", u.dtype)
    if b.dim() != dims + 1 or b.shape[:-2] != lead or b.shape[-1] != n or b.shape[-2] < 1 or width % b.shape[-2]:
        raise ValueError(f"b must be [batch{', length' if dims == 3 else ''}, groups, n] with d a multiple of groups, got shape {tuple(b.shape)}")
    _want(c, "c", u.dtype, b.shape)
    _vector(d, "d", width)
    _vector(dt_bias, "dt_bias", width)
    _same_device(u, dt=dt, a=a, b=b, c=c, d=d, z=z, dt_bias=dt_bias)
    return (width, n, b.shape[-2], _row_stride(u, "u"), _row_stride(dt, "dt"), _group_stride(b, "b"), _group_stride(c, "c"),
            _row_stride(z, "z"))


def _workspace(need, workspace, device):
    if need == 0:
        raise ValueError("unsupported shape: batch * length must stay below 2^31, and launches below 2^32 threads (of the scan: 2^24 waves)")
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _want_bytes(workspace, "workspace", need, device)
    return workspace


def ssm_scan_fwd(u, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, *, softplus=True, reset=None, lengths=None, want_saved=True, y=None,
                 h_final=None, workspace=None, stream=None):
    """Selective state space scan with its gate.  For token t, channel i (of
    group k of b and c) and state j:
        s = softplus(dt + dt_bias)   (softplus=False: the sum itself),
        h_t = exp(s a) h_{t-1} + s u b,   y = (sum_j c h_t + d u) * silu(z).

    u, dt, z [batch, length, d] BF16 or FP32 (one dtype); b, c [batch, length,
    groups, n] of that dtype; a FP32 [d, n], n up to 64; d, dt_bias FP32 [d] or
    None (0); z None: no gate; h0 FP32 [batch, d, n] or None (0).  Returns
    (y [dtype], h_final FP32, saved): saved is what the backward needs (None with
    want_saved=False), FP32 states before every 16th token."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ssm_scan_fwd(u, dt, a, b, c, d, z, dt_bias, h0, softplus=softplus, reset=reset, lengths=lengths, want_saved=want_saved, y=y,
                                h_final=h_final, workspace=workspace)
    if y is None and h_final is None and workspace is None:
        out = _native().ssm_scan_fwd(u, dt, a, b, c, d, z, dt_bias, h0, softplus, reset, lengths, want_saved, None)
        if out.__class__ is tuple:
            return out
        if out is not None:
            _check(out, "ssm_scan_fwd")
    width, n, groups, su, sdt, sb, sc, sz = _scan_args(u, dt, a, b, c, d, z, dt_bias, 3)
    batch, length, _ = u.shape
    _want(h0, "h0", _F32, (batch, width, n), optional=True)
    _dense(h0, "h0")
    _sequence_args((batch, length), reset, lengths)
    dev, given = u.device, (y, h_final)
    y = _out(y, "y", u.dtype, u.shape, dev)
    h_final = _out(h_final, "h_final", _F32, (batch, width, n), dev)
    _same_device(u, h0=h0, reset=reset, lengths=lengths, y=y, h_final=h_final)
    need = lib().ssm_scan_workspace_bytes(batch, length, width, n, groups, 0)
    workspace = _workspace(need, workspace, dev)
    saved = None
    if want_saved:
        saved = torch.empty(lib().ssm_scan_saved_bytes(batch, length, width, n, groups), dtype=torch.uint8, device=dev)
    st = lib().ssm_scan_fwd(batch, length, width, n, groups, _code(u.dtype), int(bool(softplus)), _p(u), su, _p(dt), sdt, _p(a), _p(b), sb, _p(c), sc,
                            _p(d), _p(z), sz, _p(dt_bias), _p(h0), _p(reset), _p(lengths), _p(y), _p(h_final), _p(saved), _p(workspace),
                            _nbytes(workspace), _stream(None))
    _check(st, "ssm_scan_fwd")
    _written(*given)
    return y, h_final, saved


def ssm_scan_bwd(u, dt, a, b, c, d, z, dt_bias, saved, dy, dh_final=None, *, softplus=True, reset=None, lengths=None, want_dh0=False,
                 workspace=None, stream=None):
    """Gradients of ssm_scan_fwd for the cotangents dy (of y) and dh_final (of
    h_final, None = 0), from its inputs and saved states.  Returns dict(du, ddt,
    da, db, dc, dd, dz, ddt_bias, dh0) without the keys of arguments that are
    None (dh0: unless want_dh0)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ssm_scan_bwd(u, dt, a, b, c, d, z, dt_bias, saved, dy, dh_final, softplus=softplus, reset=reset, lengths=lengths,
                                want_dh0=want_dh0, workspace=workspace)
    if workspace is None:
        out = _native().ssm_scan_bwd(u, dt, a, b, c, d, z, dt_bias, saved, dy, dh_final, softplus, reset, lengths, want_dh0, None)
        if out.__class__ is dict:
            return out
        if out is not None:
            _check(out, "ssm_scan_bwd")
    width, n, groups, su, sdt, sb, sc, sz = _scan_args(u, dt, a, b, c, d, z, dt_bias, 3)
    batch, length, _ = u.shape
    _sequence_args((batch, length), reset, lengths)
    _want(dy, "dy", u.dtype, u.shape)
    sdy = _row_stride(dy, "dy")
    _want(dh_final, "dh_final", _F32, (batch, width, n), optional=True)
    _dense(dh_final, "dh_final")
    dev = u.device
    need = lib().ssm_scan_workspace_bytes(batch, length, width, n, groups, 1)
    workspace = _workspace(need, workspace, dev)
    _want(saved, "saved", torch.uint8, (lib().ssm_scan_saved_bytes(batch, length, width, n, groups),))
    _dense(saved, "saved")
    _same_device(u, reset=reset, lengths=lengths, dy=dy, dh_final=dh_final, saved=saved)
    wide, group = dict(dtype=u.dtype, device=dev), dict(dtype=_F32, device=dev)
    out = dict(du=torch.empty(u.shape, **wide), ddt=torch.empty(u.shape, **wide), da=torch.empty(a.shape, **group),
               db=torch.empty(b.shape, **wide), dc=torch.empty(b.shape, **wide))
    if d is not None:
        out["dd"] = torch.empty(width, **group)
    if z is not None:
        out["dz"] = torch.empty(u.shape, **wide)
    if dt_bias is not None:
        out["ddt_bias"] = torch.empty(width, **group)
    if want_dh0:
        out["dh0"] = torch.empty((batch, width, n), **group)
    o = {k: _p(t) for k, t in out.items()}
    st = lib().ssm_scan_bwd(batch, length, width, n, groups, _code(u.dtype), int(bool(softplus)), _p(u), su, _p(dt), sdt, _p(a), _p(b), sb, _p(c), sc,
                            _p(d), _p(z), sz, _p(dt_bias), _p(reset), _p(lengths), _p(saved), _p(dy), sdy, _p(dh_final),
                            o["du"], o["ddt"], o["da"], o["db"], o["dc"], o.get("dd"), o.get("dz"), o.get("ddt_bias"), o.get("dh0"), _p(workspace),
                            _nbytes(workspace), _stream(None))
    _check(st, "ssm_scan_bwd")
    return out


def ssm_scan_step(h, u, dt, a, b, c, d=None, z=None, dt_bias=None, *, softplus=True, y=None, stream=None):
    """One token of `batch` sequences: the states h FP32 [batch, d, n] move on
    in place, and y [batch, d] is returned.  u, dt, z [batch, d] and b, c
    [batch, groups, n] are the token's, the rest as for ssm_scan_fwd."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ssm_scan_step(h, u, dt, a, b, c, d, z, dt_bias, softplus=softplus, y=y)
    if y is None:
        out = _native().ssm_scan_step(h, u, dt, a, b, c, d, z, dt_bias, softplus, None)
        if isinstance(out, torch.Tensor):
            return out
        if out is not None:
            _check(out, "ssm_scan_step")
    width, n, groups, su, sdt, sb, sc, sz = _scan_args(u, dt, a, b, c, d, z, dt_bias, 2)
    batch = u.shape[0]
    _want(h, "h", _F32, (batch, width, n))
    _dense(h, "h")
    given = y
    y = _out(y, "y", u.dtype, u.shape, u.device)
    _same_device(u, h=h, y=y)
    st = lib().ssm_scan_step(batch, width, n, groups, _code(u.dtype), int(bool(softplus)), _p(h), _p(u), su, _p(dt), sdt, _p(a), _p(b), sb, _p(c), sc,
                             _p(d), _p(z), sz, _p(dt_bias), _p(y), _stream(None))
    _check(st, "ssm_scan_step")
    _written(h, given)
    return y


# -------------------------------------------------------- causal convolution ---
def _conv_args(x, w, bias, act, dims):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    _want(x, "x", _DTYPES)
    if x.dim() != dims or not 1 <= x.shape[-1] <= MAX_CONV_D:
        raise ValueError(f"x must be [batch{', length' if dims == 3 else ''}, d] with d from 1 up to {MAX_CONV_D}, got shape {tuple(x.shape)}")
    d = x.shape[-1]
    _want(w, "w", _F32)
    if w.dim() != 2 or w.shape[0] != d or not 2 <= w.shape[1] <= MAX_WIDTH:
        raise ValueError(f"w must be [d, width] with width in 2..{MAX_WIDTH}, got shape {tuple(w.shape)}")
    _dense(w, "w")
    _vector(bias, "bias", d)
    _same_device(x, w=w, bias=bias)
    return d, w.shape[1], _row_stride(x, "x")


def _conv_state(state, name, x, width, optional=True):
    _want(state, name, x.dtype, (x.shape[0], width - 1, x.shape[-1]), optional=optional)
    _dense(state, name)


def causal_conv_fwd(x, w, bias=None, *, act="silu", state=None, reset=None, lengths=None, y=None, state_out=None, stream=None):
    """Short causal convolution of each channel over time:
        p_t = bias + sum_j w[:, width - 1 - j] x_{t-j},   y = p or silu(p).

    x [batch, length, d] BF16 or FP32, w FP32 [d, width] (2 to 4 taps, the last
    one the token's own), bias FP32 [d] or None.  state [batch, width - 1, d] of x's
    dtype holds the inputs from before the rows, the oldest first (None: zeros).  Returns (y,
    state_out): the inputs that the next token needs, zero where they are of an
    earlier sequence."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return causal_conv_fwd(x, w, bias, act=act, state=state, reset=reset, lengths=lengths, y=y, state_out=state_out)
    if y is None and state_out is None and act in ACTS:
        out = _native().causal_conv_fwd(x, w, bias, ACTS[act], state, reset, lengths, None)
        if out.__class__ is tuple:
            return out
        if out is not None:
            _check(out, "ssm_conv_fwd")
    d, width, sx = _conv_args(x, w, bias, act, 3)
    batch, length, _ = x.shape
    _conv_state(state, "state", x, width)
    _sequence_args((batch, length), reset, lengths)
    given = (y, state_out)
    y = _out(y, "y", x.dtype, x.shape, x.device)
    state_out = _out(state_out, "state_out", x.dtype, (batch, width - 1, d), x.device)
    _same_device(x, state=state, reset=reset, lengths=lengths, y=y, state_out=state_out)
    st = lib().ssm_conv_fwd(batch, length, d, width, _code(x.dtype), ACTS[act], _p(x), sx, _p(w), _p(bias), _p(state), _p(reset), _p(lengths), _p(y),
                            _p(state_out), _stream(None))
    _check(st, "ssm_conv_fwd")
    _written(*given)
    return y, state_out


def causal_conv_bwd(x, w, bias, dy, dstate_out=None, *, act="silu", state=None, reset=None, lengths=None, workspace=None, stream=None):
    """Gradients of causal_conv_fwd for the cotangents dy (of y) and dstate_out
    (of state_out, None = 0).  Returns dict(dx, dw, dbias, dstate) without the
    keys of arguments that are None."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return causal_conv_bwd(x, w, bias, dy, dstate_out, act=act, state=state, reset=reset, lengths=lengths, workspace=workspace)
    if workspace is None and act in ACTS:
        out = _native().causal_conv_bwd(x, w, bias, dy, dstate_out, ACTS[act], state, reset, lengths, None)
        if out.__class__ is dict:
            return out
        if out is not None:
            _check(out, "ssm_conv_bwd")
    d, width, sx = _conv_args(x, w, bias, act, 3)
    batch, length, _ = x.shape
    _conv_state(state, "state", x, width)
    _conv_state(dstate_out, "dstate_out", x, width)
    _sequence_args((batch, length), reset, lengths)
    _want(dy, "dy", x.dtype, x.shape)
    sdy = _row_stride(dy, "dy")
    workspace = _workspace(lib().ssm_conv_bwd_workspace_bytes(batch, length, d, width), workspace, x.device)
    _same_device(x, state=state, dstate_out=dstate_out, reset=reset, lengths=lengths, dy=dy)
    out = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=x.device), dw=torch.empty(w.shape, dtype=_F32, device=x.device))
    if bias is not None:
        out["dbias"] = torch.empty(d, dtype=_F32, device=x.device)
    if state is not None:
        out["dstate"] = torch.empty(state.shape, dtype=x.dtype, device=x.device)
    st = lib().ssm_conv_bwd(batch, length, d, width, _code(x.dtype), ACTS[act], _p(x), sx, _p(w), _p(bias), _p(state), _p(reset), _p(lengths), _p(dy),
                            sdy, _p(dstate_out), _p(out["dx"]), _p(out["dw"]), _p(out.get("dbias")), _p(out.get("dstate")),
                            _p(workspace), _nbytes(workspace), _stream(None))
    _check(st, "ssm_conv_bwd")
    return out


def causal_conv_step(x, w, bias, state, *, act="silu", y=None, stream=None):
    """One token x [batch, d] of `batch` sequences: state [batch, width - 1, d]
    moves on by it in place, and y [batch, d] is returned."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return causal_conv_step(x, w, bias, state, act=act, y=y)
    if y is None and act in ACTS:
        out = _native().causal_conv_step(x, w, bias, state, ACTS[act], None)
        if isinstance(out, torch.Tensor):
            return out
        if out is not None:
            _check(out, "ssm_conv_step")
    d, width, sx = _conv_args(x, w, bias, act, 2)
    _conv_state(state, "state", x, width, optional=False)
    given = y
    y = _out(y, "y", x.dtype, x.shape, x.device)
    _same_device(x, state=state, y=y)
    st = lib().ssm_conv_step(x.shape[0], d, width, _code(x.dtype), ACTS[act], _p(x), sx, _p(w), _p(bias), _p(state), _p(y), _stream(None))
    _check(st, "ssm_conv_step")
    _written(state, given)
    return y
