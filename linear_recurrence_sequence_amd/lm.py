"""Language-model operators around the recurrent mixers: thin Python binding
of the C ABI in include/lm_ops.h.

Block norms with their gate and residual scale, the softmax cross entropy of a
linear head, the AdamW step over many tensors, and the embedding lookup.  Argument checks and
marshalling only: every step runs in the HIP kernels of libsamu_scan.so, on
the current stream or the one given.  The differentiable forms are in
autograd.py.

With a stream given a call runs as if that stream were the current one: its
outputs and workspace are allocated there.  Tensors lie on the current device,
or the stream's.

A plainly right call with outputs of its own goes through _lm_bind (see
csrc/lm_bind.cpp), which makes the checks below in a few microseconds; every other call is
checked, and where it is wrong refused, here.
"""
import ctypes

import torch

from . import scan
from .scan import _check, _code, _nbytes, _stream, _want, _want_bytes

_BF16, _F32 = torch.bfloat16, torch.float32
_DTYPES = (_BF16, _F32)
GATES = {"none": 0, "sigmoid": 1, "silu": 2}
ADAMW_BLOCK = 256
EMBED_MAX_D = 1 << 23

_lib = None
_bound = None


def _native():
    """The module behind the usual calls (raises if it has not been built)."""
    global _bound
    if _bound is None:
        scan.lib()
        from . import _lm_bind
        _lm_bind.setup(torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
        _bound = _lm_bind
    return _bound


def lib():
    """The loaded library with the argument types of lm_ops.h."""
    global _lib
    if _lib is not None:
        return _lib
    L = scan.lib()
    i, i64, sz, vp, dbl = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_double
    L.lm_block_norm_fwd.argtypes = [i64, i, i, i, i, dbl] + [vp, i64] * 3 + [vp] * 6 + [vp]
    L.lm_block_norm_fwd.restype = i
    L.lm_block_norm_bwd_workspace_bytes.argtypes = [i64, i]
    L.lm_block_norm_bwd_workspace_bytes.restype = sz
    L.lm_block_norm_bwd.argtypes = [i64, i, i, i, i] + [vp, i64] * 3 + [vp] * 4 + [vp, i64] * 2 + [vp] * 6 + [vp, sz, vp]
    L.lm_block_norm_bwd.restype = i
    L.lm_linear_ce_workspace_bytes.argtypes = [i64, i, i64, i]
    L.lm_linear_ce_workspace_bytes.restype = sz
    L.lm_linear_ce_fwd.argtypes = [i64, i, i64, dbl, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    L.lm_linear_ce_fwd.restype = i
    L.lm_linear_ce_bwd.argtypes = [i64, i, i64, dbl, vp, i64] + [vp] * 7 + [i, vp, sz, vp]
    L.lm_linear_ce_bwd.restype = i
    L.lm_adamw_step.argtypes = [i, i, i, i] + [vp] * 9 + [dbl] * 4 + [i64, vp]
    L.lm_adamw_step.restype = i
    L.lm_embed_fwd.argtypes = [i64, i, i64, i, i, dbl, vp, vp, vp, vp]
    L.lm_embed_fwd.restype = i
    L.lm_embed_bwd_workspace_bytes.argtypes = [i64, i, i64]
    L.lm_embed_bwd_workspace_bytes.restype = sz
    L.lm_embed_bwd.argtypes = [i64, i, i64, i, i, dbl, vp, vp, i64, i, vp, vp, sz, vp]
    L.lm_embed_bwd.restype = i
    _lib = L
    return L


def _p(t):
    """Address of a device tensor (its strides were checked by the caller)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    return t.data_ptr()


def _current(device):
    """Refuses tensors of another device than the current one: the launch and its stream are the current one's."""
    if device.type == "cuda" and device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}: call under "
                         f"torch.cuda.device, or with a stream of {device}")


def _same_device(first, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")
    _current(first.device)


def _written(*tensors):
    """Says to autograd that a call wrote tensors of the caller's: a graph that kept one refuses its backward."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None and not t.is_inference()])


def _dense(t, name):
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _row_stride(t, name):
    """Elements from one row of t [..., d] to the next; refuses what is not
    rows of dense columns at one distance."""
    if t is None:
        return 0
    if t.is_contiguous():
        return t.shape[-1]
    d = t.shape[-1]
    if t.stride(-1) != 1 and d > 1:
        raise ValueError(f"{name} must have dense columns (stride 1 along its last dimension)")
    step = None          # of the innermost leading dimension longer than one
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step, reach = s, s * n
        elif s != reach:
            raise ValueError(f"{name} must have its rows at one distance (got strides {t.stride()})")
        else:
            reach = s * n
    return d if step is None else step


# ------------------------------------------------------------- block norms ---
def _norm_args(x, y, gate, w_post, scale, w_pre, gate_act):
    if gate_act not in GATES:
        raise ValueError(f"gate_act must be one of {sorted(GATES)}, got {gate_act!r}")
    _want(x, "x", _DTYPES)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must be [..., d] with d >= 1, got shape {tuple(x.shape)}")
    shape, d = x.shape, x.shape[-1]
    _want(y, "y", _DTYPES, shape)
    if (gate is None) != (gate_act == "none"):
        raise ValueError("a gate is given with, and only with, a gate activation")
    _want(gate, "gate", y.dtype, shape, optional=True)
    if (w_post is None) != (scale is None):
        raise ValueError("w_post and scale are given together or not at all")
    _want(w_post, "w_post", _F32, (d,), optional=True)
    _want(scale, "scale", _F32, (d,), optional=True)
    _want(w_pre, "w_pre", _F32, (d,))
    for t, n in ((w_post, "w_post"), (scale, "scale"), (w_pre, "w_pre")):
        _dense(t, n)
    _same_device(x, y=y, gate=gate, w_post=w_post, scale=scale, w_pre=w_pre)
    return x.numel() // d, d, _row_stride(x, "x"), _row_stride(y, "y"), _row_stride(gate, "gate")


def block_norm_fwd(x, y, gate, w_post, scale, w_pre, *, eps=1e-6, gate_act="none", r=None, n=None, stats=None,
                   stream=None):
    """Adds a block's output to the residual stream and norms the sum for the
    next block:
        r = x + scale * act(gate) * norm(y) * w_post,   n = norm(r) * w_pre
    with norm(v) = v / sqrt(mean(v^2) + eps) over the last dimension; without
    w_post and scale, r = x + act(gate) * y.

    x [..., d] BF16 or FP32 (the stream), y and gate [..., d] BF16 or FP32 (the
    branch); rows may lie apart (views of a wider projection).  gate_act is
    "none" (gate None), "sigmoid" or "silu"; weights are FP32 [d].  r may be x
    itself (not before a backward, which reads x as it was).  Returns (r [stream dtype], n [branch dtype], stats f32 [rows, 2])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return block_norm_fwd(x, y, gate, w_post, scale, w_pre, eps=eps, gate_act=gate_act, r=r, n=n, stats=stats)
    if r is None and n is None and stats is None and gate_act in GATES:
        out = _native().block_norm_fwd(x, y, gate, w_post, scale, w_pre, eps, GATES[gate_act], None)
        if out.__class__ is tuple:
            return out
        if out is not None:
            _check(out, "lm_block_norm_fwd")
    rows, d, sx, sy, sg = _norm_args(x, y, gate, w_post, scale, w_pre, gate_act)
    dev, given = x.device, (r, n, stats)
    if r is None:
        r = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _want(r, "r", x.dtype, x.shape)
        _dense(r, "r")
    if n is None:
        n = torch.empty(x.shape, dtype=y.dtype, device=dev)
    else:
        _want(n, "n", y.dtype, x.shape)
        _dense(n, "n")
    if stats is None:
        stats = torch.empty((rows, 2), dtype=_F32, device=dev)
    else:
        _want(stats, "stats", _F32, (rows, 2))
        _dense(stats, "stats")
    _same_device(x, r=r, n=n, stats=stats)
    st = lib().lm_block_norm_fwd(rows, d, _code(x.dtype), _code(y.dtype), GATES[gate_act], eps, _p(x),
                                 sx, _p(y), sy, _p(gate), sg, _p(w_post), _p(scale), _p(w_pre), _p(r), _p(n),
                                 _p(stats), _stream(None))
    _check(st, "lm_block_norm_fwd")
    _written(*given)
    return r, n, stats


def block_norm_bwd(x, y, gate, w_post, scale, w_pre, stats, dr, dn, *, eps=1e-6, gate_act="none", workspace=None,
                   stream=None):
    """Gradients of block_norm_fwd for the cotangents dr (of r, stream dtype)
    and dn (of n, branch dtype); either may be None (zero).  stats are the
    forward's (they hold eps's part).  Returns dict(dx, dy, dgate, dw_post,
    dscale, dw_pre) without the keys of arguments that are None."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return block_norm_bwd(x, y, gate, w_post, scale, w_pre, stats, dr, dn, eps=eps, gate_act=gate_act, workspace=workspace)
    if workspace is None and gate_act in GATES:
        out = _native().block_norm_bwd(x, y, gate, w_post, scale, w_pre, stats, dr, dn, GATES[gate_act], None)
        if out.__class__ is dict:
            return out
        if out is not None:
            _check(out, "lm_block_norm_bwd")
    rows, d, sx, sy, sg = _norm_args(x, y, gate, w_post, scale, w_pre, gate_act)
    _want(stats, "stats", _F32, (rows, 2))
    _dense(stats, "stats")
    _want(dr, "dr", x.dtype, x.shape, optional=True)
    _want(dn, "dn", y.dtype, x.shape, optional=True)
    _same_device(x, stats=stats, dr=dr, dn=dn)
    dev = x.device
    out = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=dev), dy=torch.empty(x.shape, dtype=y.dtype, device=dev))
    if gate is not None:
        out["dgate"] = torch.empty(x.shape, dtype=y.dtype, device=dev)
    for k, w in (("dw_post", w_post), ("dscale", scale), ("dw_pre", w_pre)):
        if w is not None:
            out[k] = torch.empty(d, dtype=_F32, device=dev)
    need = lib().lm_block_norm_bwd_workspace_bytes(rows, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _want_bytes(workspace, "workspace", need, dev)
    st = lib().lm_block_norm_bwd(rows, d, _code(x.dtype), _code(y.dtype), GATES[gate_act], _p(x), sx,
                                 _p(y), sy, _p(gate), sg, _p(w_post), _p(scale), _p(w_pre), _p(stats), _p(dr),
                                 _row_stride(dr, "dr"), _p(dn), _row_stride(dn, "dn"), _p(out["dx"]), _p(out["dy"]),
                                 _p(out.get("dgate")), _p(out.get("dw_post")), _p(out.get("dscale")),
                                 _p(out["dw_pre"]), _p(workspace), _nbytes(workspace), _stream(None))
    _check(st, "lm_block_norm_bwd")
    return out


# ---------------------------------------------------- linear cross entropy ---
def _ce_args(h, w, target):
    _want(h, "h", _BF16)
    _want(w, "w", _BF16)
    if h.dim() < 1 or w.dim() != 2 or h.shape[-1] != w.shape[1]:
        raise ValueError(f"h must be [..., d] and w [v, d], got shapes {tuple(h.shape)} and {tuple(w.shape)}")
    _want(target, "target", torch.int64, h.shape[:-1])
    _dense(w, "w")
    _dense(target, "target")
    _same_device(h, w=w, target=target)
    return target.numel(), w.shape[1], w.shape[0], _row_stride(h, "h")


def _ce_workspace(n, d, v, backward, workspace, dev):
    need = lib().lm_linear_ce_workspace_bytes(n, d, v, backward)
    if need == 0:
        raise ValueError(f"unsupported shape: {n} tokens, width {d}, vocabulary {v} (the width must be a multiple of 8 in 8..65536)")
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _want_bytes(workspace, "workspace", need, dev)
    return workspace


def linear_ce_fwd(h, w, target, *, softcap=0.0, loss=None, lse=None, workspace=None, stream=None):
    """Cross entropy of a linear head, token by token, without its logits:
        z = h w^T (softcap > 0: softcap * tanh(z / softcap)),
        lse = logsumexp(z),  loss = lse - z[target].

    h [..., d] BF16 (rows may lie apart, 16-byte aligned), w [v, d] BF16, target
    [...] int64; a negative target does not count (loss 0).  Returns (loss, lse)
    FP32 [...]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_ce_fwd(h, w, target, softcap=softcap, loss=loss, lse=lse, workspace=workspace)
    if loss is None and lse is None and workspace is None:
        out = _native().linear_ce_fwd(h, w, target, softcap, None)
        if out.__class__ is tuple:
            return out
        if out is not None:
            _check(out, "lm_linear_ce_fwd")
    n, d, v, sh = _ce_args(h, w, target)
    dev, given = h.device, (loss, lse)
    out = []
    for t, name in ((loss, "loss"), (lse, "lse")):
        if t is None:
            t = torch.empty(target.shape, dtype=_F32, device=dev)
        else:
            _want(t, name, _F32, target.shape)
            _dense(t, name)
        out.append(t)
    loss, lse = out
    workspace = _ce_workspace(n, d, v, 0, workspace, dev)
    st = lib().lm_linear_ce_fwd(n, d, v, softcap, _p(h), sh, _p(w), _p(target), _p(loss), _p(lse), _p(workspace),
                                _nbytes(workspace), _stream(None))
    _check(st, "lm_linear_ce_fwd")
    _written(*given)
    return loss, lse


def linear_ce_bwd(h, w, target, lse, dloss, dlse=None, *, softcap=0.0, grad_dtype=_BF16, dh=None, dw=None,
                  workspace=None, stream=None):
    """Gradients of linear_ce_fwd for the cotangents dloss and dlse (FP32, as
    the target; dlse None = 0), from its lse.  Returns dict(dh, dw) of
    grad_dtype.

    The cotangent of the logits, dz, is rounded to BF16 for the two products, whose operands are BF16 and whose sums
    are FP32, whatever grad_dtype is: a term of dh and dw is off by up to 2^-8 of itself, and FP32 gradients save the
    last rounding alone.  BF16 gradients of 2048 tokens x 1024 x 32000 are 0.0019 of their size from 64 bits, with dz in FP32 0.0017."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_ce_bwd(h, w, target, lse, dloss, dlse, softcap=softcap, grad_dtype=grad_dtype, dh=dh, dw=dw, workspace=workspace)
    if dh is None and dw is None and workspace is None and grad_dtype in _DTYPES:
        out = _native().linear_ce_bwd(h, w, target, lse, dloss, dlse, softcap, grad_dtype is _F32, None)
        if out.__class__ is dict:
            return out
        if out is not None:
            _check(out, "lm_linear_ce_bwd")
    n, d, v, sh = _ce_args(h, w, target)
    dev = h.device
    for t, name in ((lse, "lse"), (dloss, "dloss"), (dlse, "dlse")):
        _want(t, name, _F32, target.shape, optional=name == "dlse")
        _dense(t, name)
    _code(grad_dtype)
    given = (dh, dw)
    if dh is None:
        dh = torch.empty(h.shape, dtype=grad_dtype, device=dev)
    if dw is None:
        dw = torch.empty(w.shape, dtype=dh.dtype, device=dev)
    for t, name, shape in ((dh, "dh", h.shape), (dw, "dw", w.shape)):
        _want(t, name, _DTYPES if name == "dh" else dh.dtype, shape)
        _dense(t, name)
    _same_device(h, lse=lse, dloss=dloss, dlse=dlse, dh=dh, dw=dw)
    workspace = _ce_workspace(n, d, v, 1, workspace, dev)
    st = lib().lm_linear_ce_bwd(n, d, v, softcap, _p(h), sh, _p(w), _p(target), _p(lse), _p(dloss), _p(dlse), _p(dh),
                                _p(dw), _code(dh.dtype), _p(workspace), _nbytes(workspace), _stream(None))
    _check(st, "lm_linear_ce_bwd")
    _written(*given)
    return dict(dh=dh, dw=dw)


# ------------------------------------------------------------------- AdamW ---
_F8 = torch.float8_e4m3fn


def _adamw_list(ts, name, count, dtype, sizes, device):
    if len(ts) != count:
        raise ValueError(f"{name} holds {len(ts)} tensors, expected {count}")
    for i, (t, k) in enumerate(zip(ts, sizes)):
        if t.dtype != dtype or t.numel() != k or t.device != device or not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be a contiguous {dtype} tensor of {k} elements on {device}, got "
                             f"{t.dtype}, {t.numel()} elements, strides {t.stride()}, {t.device}")
    return (ctypes.c_void_p * count)(*[t.data_ptr() for t in ts])


def adamw_step(params, grads, m, v, *, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, masters=None,
               m_scales=None, v_scales=None, stream=None):
    """One AdamW step over many tensors, in place, in one launch per 48 tensors.

    params, grads: lists of BF16 or FP32 tensors (one dtype a list); m, v: FP32
    moments, or (with m_scales and v_scales) float8_e4m3fn codes whose blocks of
    256 consecutive elements have one FP32 scale each, v's codes holding the
    square root (see adamw_state).  masters: FP32 weights of which params are
    the rounded copies.  weight_decay: a number, or one a tensor.  step counts
    from 1; it and lr are taken by value, so a captured graph repeats them."""
    st = _native().adamw_step(params, grads, m, v, masters, m_scales, v_scales, weight_decay, step, lr, betas[0], betas[1], eps, stream)
    if st is not None:
        _check(st, "lm_adamw_step")
        return
    count = len(params)
    decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * count
    if len(decay) != count:
        raise ValueError(f"weight_decay holds {len(decay)} numbers, expected {count}")
    if (m_scales is None) != (v_scales is None):
        raise ValueError("m_scales and v_scales are given together or not at all")
    if len(grads) != count or len(m) != count or len(v) != count:
        raise ValueError(f"params, grads, m and v must be as long as each other, got {count}, {len(grads)}, "
                         f"{len(m)}, {len(v)}")
    if count == 0:
        return
    p0, g0 = params[0], grads[0]
    _want(p0, "params[0]", _DTYPES)
    _want(g0, "grads[0]", _DTYPES)
    dev, bits = p0.device, 32 if m_scales is None else 8
    sizes = [t.numel() for t in params]
    state = _F32 if bits == 32 else _F8
    args = [_adamw_list(params, "params", count, p0.dtype, sizes, dev),
            _adamw_list(grads, "grads", count, g0.dtype, sizes, dev),
            _adamw_list(m, "m", count, state, sizes, dev), _adamw_list(v, "v", count, state, sizes, dev),
            None if masters is None else _adamw_list(masters, "masters", count, _F32, sizes, dev)]
    if bits == 8:
        blocks = [-(-k // ADAMW_BLOCK) for k in sizes]
        args += [_adamw_list(m_scales, "m_scales", count, _F32, blocks, dev),
                 _adamw_list(v_scales, "v_scales", count, _F32, blocks, dev)]
    else:
        args += [None, None]
    if not p0.is_cuda:
        raise ValueError("expected device tensors")
    if stream is not None:
        with torch.cuda.stream(stream):
            return adamw_step(params, grads, m, v, step=step, lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, masters=masters,
                              m_scales=m_scales, v_scales=v_scales)
    _current(dev)
    st = lib().lm_adamw_step(count, _code(p0.dtype), _code(g0.dtype), bits, *args, (ctypes.c_int64 * count)(*sizes),
                             (ctypes.c_double * count)(*decay), lr, betas[0], betas[1], eps, int(step),
                             _stream(None))
    _check(st, "lm_adamw_step")
    _written(*params)


def adamw_state(p, bits=32):
    """Zero moments for a parameter: dict(m, v) in FP32, or dict(m, v, m_scale,
    v_scale) in 8 bits."""
    if bits == 32:
        return dict(m=torch.zeros(p.shape, dtype=_F32, device=p.device), v=torch.zeros(p.shape, dtype=_F32, device=p.device))
    if bits != 8:
        raise ValueError("bits must be 8 or 32")
    blocks = -(-p.numel() // ADAMW_BLOCK)
    z = dict(dtype=torch.uint8, device=p.device)
    s = dict(dtype=_F32, device=p.device)
    return dict(m=torch.zeros(p.shape, **z).view(_F8), v=torch.zeros(p.shape, **z).view(_F8),
                m_scale=torch.zeros(blocks, **s), v_scale=torch.zeros(blocks, **s))


# -------------------------------------------------------- embedding lookup ---
def embed_fwd(tokens, w, *, scale=1.0, out_dtype=None, out=None, stream=None):
    """Rows of an embedding: out_t = scale * w[tokens_t].

    tokens [...] int64, w [v, d] BF16 or FP32.  A negative token is padding: its
    row of out is zero (a token >= v: NaN).  out_dtype: BF16 or FP32, w's if
    None.  Returns out [..., d]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed_fwd(tokens, w, scale=scale, out_dtype=out_dtype, out=out)
    if out is None and (out_dtype is None or out_dtype in _DTYPES):
        r = _native().embed_fwd(tokens, w, scale, None if out_dtype is None else out_dtype is _F32, None)
        if isinstance(r, torch.Tensor):
            return r
        if r is not None:
            _check(r, "lm_embed_fwd")
    _want(tokens, "tokens", torch.int64)
    _want(w, "w", _DTYPES)
    if w.dim() != 2 or w.shape[0] < 1 or not 1 <= w.shape[1] <= EMBED_MAX_D:
        raise ValueError(f"w must be [v, d] with v >= 1 and d from 1 up to {EMBED_MAX_D}, got shape {tuple(w.shape)}")
    _dense(tokens, "tokens")
    _dense(w, "w")
    v, d = w.shape
    given = out
    if out_dtype is None:
        out_dtype = w.dtype if out is None else out.dtype
    _code(out_dtype)
    if out is None:
        out = torch.empty((*tokens.shape, d), dtype=out_dtype, device=w.device)
    _want(out, "out", out_dtype, (*tokens.shape, d))
    _dense(out, "out")
    _same_device(w, tokens=tokens, out=out)
    st = lib().lm_embed_fwd(tokens.numel(), d, v, _code(w.dtype), _code(out_dtype), scale, _p(tokens), _p(w), _p(out), _stream(None))
    _check(st, "lm_embed_fwd")
    _written(given)
    return out


def embed_bwd(tokens, dout, v, *, scale=1.0, grad_dtype=_BF16, dw=None, accumulate=False, workspace=None, stream=None):
    """Gradient of embed_fwd's w [v, d] for the cotangent dout [..., d] (BF16 or
    FP32; rows may lie apart): dw_j = scale * the sum of dout over the tokens j,
    FP32 sums in an order that the tokens alone decide, rounded once.  dw is of
    grad_dtype, zero where no token is.  accumulate: the sums are added to the dw given, before the
    rounding; rows without tokens stay as they are.  Returns dw."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed_bwd(tokens, dout, v, scale=scale, grad_dtype=grad_dtype, dw=dw, accumulate=accumulate, workspace=workspace)
    if dw is None and workspace is None and not accumulate and grad_dtype in _DTYPES:
        r = _native().embed_bwd(tokens, dout, v, scale, grad_dtype is _F32, None)
        if isinstance(r, torch.Tensor):
            return r
        if r is not None:
            _check(r, "lm_embed_bwd")
    _want(tokens, "tokens", torch.int64)
    _want(dout, "dout", _DTYPES)
    if dout.dim() < 1 or dout.shape[:-1] != tokens.shape or not 1 <= dout.shape[-1] <= EMBED_MAX_D:
        raise ValueError(f"dout must be [..., d] with the tokens' shape in front and d from 1 up to {EMBED_MAX_D}, "
                         f"got shapes {tuple(dout.shape)} and {tuple(tokens.shape)}")
    _dense(tokens, "tokens")
    n, d, v, sg = tokens.numel(), dout.shape[-1], int(v), _row_stride(dout, "dout")
    if accumulate and dw is None:
        raise ValueError("accumulate needs a dw to add to")
    given = dw
    if dw is None:
        if v < 1:
            raise ValueError(f"v must be at least 1, got {v}")
        _code(grad_dtype)
        dw = torch.empty((v, d), dtype=grad_dtype, device=dout.device)
    _want(dw, "dw", _DTYPES, (v, d))
    _dense(dw, "dw")
    _same_device(dout, tokens=tokens, dw=dw)
    need = lib().lm_embed_bwd_workspace_bytes(n, d, v)
    if need == 0:
        raise ValueError(f"unsupported shape: {n} tokens, width {d}, vocabulary {v}")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dout.device)
    _want_bytes(workspace, "workspace", need, dout.device)
    st = lib().lm_embed_bwd(n, d, v, _code(dout.dtype), _code(dw.dtype), scale, _p(tokens), _p(dout), sg, int(bool(accumulate)),
                            _p(dw), _p(workspace), _nbytes(workspace), _stream(None))
    _check(st, "lm_embed_bwd")
    _written(given)
    return dw
