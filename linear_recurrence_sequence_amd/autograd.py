"""The scans, the projections and the language-model operators as differentiable torch operations.

Each forward calls the library's forward entry point and keeps its saved
record (a uint8 tensor) for the backward; each backward calls the adjoint
entry point.  Nothing here computes: these classes only route tensors to the
C ABI.  Gradients come back in the dtypes of the inputs they belong to (BF16
streams in BF16, FP32 parameters in FP32, BF16 projection weights in BF16).
An output whose gradient is not needed passes a NULL cotangent (zero) to the
library.  The streams (x_sel, b; x, l^x, l^a) must be BF16, the library's
input format: a tensor of another dtype is refused rather than converted."""
import torch

from . import lm, scan, ssm


def _need_bf16(**tensors):
    for name, t in tensors.items():
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be torch.bfloat16 (the scan's input format), got {t.dtype}")


class SamuScan(torch.autograd.Function):
    """SAMU mixer scan: (x_sel, b, w_phi, w_r, a_phi, a_r, nu, theta, z0) ->
    (y [B, L, D/2, 2] BF16, z_final [B, D/2, 2] FP32)."""

    @staticmethod
    def forward(ctx, x_sel, b, w_phi, w_r, a_phi, a_r, nu, theta, z0, K, G):
        _need_bf16(x_sel=x_sel, b=b)
        y, z_final, saved = scan.samu_scan_fwd(x_sel, b, w_phi, w_r, a_phi, a_r, nu, theta, z0, K=K, G=G,
                                               y_dtype=torch.bfloat16)
        ctx.save_for_backward(x_sel, b, w_phi, w_r, a_phi, a_r, nu, theta, saved)
        ctx.K, ctx.G, ctx.has_z0 = K, G, z0 is not None
        ctx.set_materialize_grads(False)
        return y, z_final

    @staticmethod
    def backward(ctx, dy, dz_final):
        x_sel, b, w_phi, w_r, a_phi, a_r, nu, theta, saved = ctx.saved_tensors
        B, L, D = x_sel.shape
        if dy is None:
            dy = torch.zeros((B, L, D // 2, 2), dtype=torch.bfloat16, device=b.device)
        dy = dy.to(torch.bfloat16).contiguous()
        dzf = None if dz_final is None else dz_final.float().contiguous()
        g = scan.samu_scan_bwd(x_sel, b, w_phi, w_r, a_phi, a_r, nu, theta, saved, dy, dzf, K=ctx.K, G=ctx.G,
                               grad_dtype=torch.bfloat16, want_dz0=ctx.has_z0)
        return (g["dx_sel"], g["db"], g["dw_phi"], g["dw_r"], g["da_phi"], g["da_r"], g["dnu"],
                g["dtheta"], g["dz0"] if ctx.has_z0 else None, None, None)


class RglruScan(torch.autograd.Function):
    """RG-LRU scan: (x, lx, la, alpha, reset, h0) -> (y [B, L, D] BF16,
    h_final [B, D] FP32); `reset` (uint8 [B, L] or None) takes no
    gradient."""

    @staticmethod
    def forward(ctx, x, lx, la, alpha, reset, h0, K, G):
        _need_bf16(x=x, lx=lx, la=la)
        y, h_final, saved = scan.rglru_scan_fwd(x, lx, la, alpha, reset, h0, K=K, G=G, y_dtype=torch.bfloat16)
        ctx.save_for_backward(x, lx, la, alpha, reset, saved)
        ctx.K, ctx.G, ctx.has_h0 = K, G, h0 is not None
        ctx.set_materialize_grads(False)
        return y, h_final

    @staticmethod
    def backward(ctx, dy, dh_final):
        x, lx, la, alpha, reset, saved = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        dy = dy.to(torch.bfloat16).contiguous()
        dhf = None if dh_final is None else dh_final.float().contiguous()
        g = scan.rglru_scan_bwd(x, lx, la, alpha, reset, saved, dy, dhf, K=ctx.K, G=ctx.G,
                                grad_dtype=torch.bfloat16, want_dh0=ctx.has_h0)
        return (g["dx"], g["dlx"], g["dla"], g["dalpha"], None,
                g["dh0"] if ctx.has_h0 else None, None, None)


class RglruGateProj(torch.autograd.Function):
    """The two 16-block block-diagonal gate projections: (x, w_x, b_x, w_a,
    b_a) -> (l^x, l^a), BF16 [B, L, D]."""

    @staticmethod
    def forward(ctx, x, w_x, b_x, w_a, b_a):
        _need_bf16(x=x, w_x=w_x, w_a=w_a)
        lx, la = scan.rglru_gate_proj_fwd(x, w_x, b_x, w_a, b_a)
        ctx.save_for_backward(x, w_x, w_a)
        ctx.set_materialize_grads(False)
        return lx, la

    @staticmethod
    def backward(ctx, dlx, dla):
        x, w_x, w_a = ctx.saved_tensors
        ref = dlx if dlx is not None else dla
        if ref is None:
            return None, None, None, None, None
        dt = torch.float32 if ref.dtype == torch.float32 else torch.bfloat16  # the adjoint's cotangent types
        z = None
        if dlx is None or dla is None:
            z = torch.zeros(x.shape, dtype=dt, device=x.device)
        dlx = z if dlx is None else dlx.to(dt).contiguous()
        dla = z if dla is None else dla.to(dt).contiguous()
        g = scan.rglru_gate_proj_bwd(x, w_x, w_a, dlx, dla, torch.zeros(x.shape, dtype=dt, device=x.device))
        return (g["dx"].to(x.dtype), g["dw_x"].to(w_x.dtype), g["db_x"], g["dw_a"].to(w_a.dtype), g["db_a"])


def samu_scan(x_sel, b, w_phi, w_r, a_phi, a_r, nu, theta, z0=None, *, K=32, G=0):
    return SamuScan.apply(x_sel, b, w_phi, w_r, a_phi, a_r, nu, theta, z0, K, G)


def rglru_scan(x, lx, la, alpha, reset=None, h0=None, *, K=16, G=0):
    return RglruScan.apply(x, lx, la, alpha, reset, h0, K, G)


def rglru_gate_proj(x, w_x, b_x, w_a, b_a):
    return RglruGateProj.apply(x, w_x, b_x, w_a, b_a)


class RglruLayer(torch.autograd.Function):
    """Input to output of the RG-LRU layer as one differentiable operation:
    the two gate projections, then the scan.  x feeds both, so its gradient
    has two terms: the backward runs the scan adjoint with FP32 cotangents,
    accumulates the projection adjoint into that FP32 dx in place (the
    library's dx_in accumulate), and rounds the sum to BF16 once."""

    @staticmethod
    def forward(ctx, x, w_x, b_x, w_a, b_a, alpha, reset, h0, K, G):
        _need_bf16(x=x, w_x=w_x, w_a=w_a)
        lx, la = scan.rglru_gate_proj_fwd(x, w_x, b_x, w_a, b_a)
        y, h_final, saved = scan.rglru_scan_fwd(x, lx, la, alpha, reset, h0, K=K, G=G, y_dtype=torch.bfloat16)
        ctx.save_for_backward(x, w_x, w_a, lx, la, alpha, reset, saved)
        ctx.K, ctx.G, ctx.has_h0 = K, G, h0 is not None
        ctx.set_materialize_grads(False)
        return y, h_final

    @staticmethod
    def backward(ctx, dy, dh_final):
        x, w_x, w_a, lx, la, alpha, reset, saved = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        dy = dy.to(torch.bfloat16).contiguous()
        dhf = None if dh_final is None else dh_final.float().contiguous()
        g = scan.rglru_scan_bwd(x, lx, la, alpha, reset, saved, dy, dhf, K=ctx.K, G=ctx.G,
                                grad_dtype=torch.float32, want_dh0=ctx.has_h0)
        p = scan.rglru_gate_proj_bwd(x, w_x, w_a, g["dlx"], g["dla"], g["dx"], dx_out=g["dx"])
        return (p["dx"].to(torch.bfloat16), p["dw_x"].to(w_x.dtype), p["db_x"], p["dw_a"].to(w_a.dtype),
                p["db_a"], g["dalpha"], None, g["dh0"] if ctx.has_h0 else None, None, None)


def rglru_layer(x, w_x, b_x, w_a, b_a, alpha, reset=None, h0=None, *, K=16, G=0):
    """Input to output of the RG-LRU layer: gate projections, then the scan
    (one autograd node; x's gradient is rounded to BF16 once)."""
    return RglruLayer.apply(x, w_x, b_x, w_a, b_a, alpha, reset, h0, K, G)


class _Once(torch.autograd.Function):
    """A gradient as it is, tied to all that it was formed from: differentiating it raises, where it would otherwise count as a
    constant.  (torch's once_differentiable looks at the cotangents alone, which need not depend on anything.)"""

    @staticmethod
    def forward(ctx, what, grad, *formed_from):
        ctx.what = what
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError(f"{ctx.what} has no second derivative")


def _once(what, grads, *formed_from):
    """The gradients of a backward, refused a derivative of their own where create_graph asks for one."""
    if not torch.is_grad_enabled():
        return grads
    return tuple(None if g is None else _Once.apply(what, g, *formed_from) for g in grads)


class BlockNorm(torch.autograd.Function):
    """Residual sum and norms around a block: (x, y, gate, w_post, scale,
    w_pre) -> (r, n), as lm.block_norm_fwd.  A second derivative raises."""

    @staticmethod
    def forward(ctx, x, y, gate, w_post, scale, w_pre, eps, gate_act):
        r, n, stats = lm.block_norm_fwd(x, y, gate, w_post, scale, w_pre, eps=eps, gate_act=gate_act)
        ctx.save_for_backward(x, y, gate, w_post, scale, w_pre, stats)
        ctx.eps, ctx.gate_act = eps, gate_act
        ctx.set_materialize_grads(False)
        return r, n

    @staticmethod
    def backward(ctx, dr, dn):
        x, y, gate, w_post, scale, w_pre, stats = ctx.saved_tensors
        # expanded cotangents (of a sum) have no rows to read: lay them out
        dr = None if dr is None else dr.contiguous()
        dn = None if dn is None else dn.contiguous()
        g = lm.block_norm_bwd(x, y, gate, w_post, scale, w_pre, stats, dr, dn, eps=ctx.eps, gate_act=ctx.gate_act)
        grads = (g["dx"], g["dy"], g.get("dgate"), g.get("dw_post"), g.get("dscale"), g["dw_pre"])
        return (*_once("block_norm", grads, x, y, gate, w_post, scale, w_pre, dr, dn), None, None)


def block_norm(x, y, gate, w_post, scale, w_pre, *, eps=1e-6, gate_act="none"):
    """r = x + scale * act(gate) * norm(y) * w_post and n = norm(r) * w_pre
    (without w_post and scale: r = x + act(gate) * y); returns (r, n)."""
    return BlockNorm.apply(x, y, gate, w_post, scale, w_pre, eps, gate_act)


class LinearCe(torch.autograd.Function):
    """Softmax cross entropy of a linear head: (h, w, target) -> (loss, lse),
    token by token, as lm.linear_ce_fwd.  A second derivative raises."""

    @staticmethod
    def forward(ctx, h, w, target, softcap):
        loss, lse = lm.linear_ce_fwd(h, w, target, softcap=softcap)
        ctx.save_for_backward(h, w, target, lse)
        ctx.softcap = softcap
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, dlse):
        h, w, target, lse = ctx.saved_tensors
        if dloss is None:
            dloss = torch.zeros_like(lse)
        g = lm.linear_ce_bwd(h, w, target, lse, dloss.float().contiguous(), None if dlse is None else dlse.float().contiguous(),
                             softcap=ctx.softcap)
        return (*_once("linear_ce", (g["dh"], g["dw"]), h, w, dloss, dlse), None, None)


def linear_ce(h, w, target, *, softcap=0.0):
    """Token-wise cross entropy of the logits h w^T (capped where softcap > 0),
    which are not kept; returns (loss, lse).  Negative targets do not count.
    The backward rounds the logits' cotangent to BF16 for its two products."""
    return LinearCe.apply(h, w, target, softcap)


class Embed(torch.autograd.Function):
    """Embedding lookup: w -> out, as lm.embed_fwd.  A second derivative raises."""

    @staticmethod
    def forward(ctx, tokens, w, scale, out_dtype):
        ctx.save_for_backward(tokens)
        ctx.v, ctx.scale, ctx.dtype = w.shape[0], scale, w.dtype
        return lm.embed_fwd(tokens, w, scale=scale, out_dtype=out_dtype)

    @staticmethod
    def backward(ctx, dout):
        tokens, = ctx.saved_tensors
        dw = lm.embed_bwd(tokens, dout.contiguous(), ctx.v, scale=ctx.scale, grad_dtype=ctx.dtype)
        return (None, *_once("embed", (dw,), dout), None, None)


def embed(tokens, w, *, scale=1.0, out_dtype=None):
    """Rows of an embedding, scale * w[tokens]; a negative token's row is zero.
    The gradient is dense, summed in a fixed order."""
    return Embed.apply(tokens, w, scale, out_dtype)


class SsmScan(torch.autograd.Function):
    """Selective scan: (u, dt, a, b, c, d, z, dt_bias, h0) -> (y, h_final), as
    ssm.ssm_scan_fwd.  A second derivative raises."""

    @staticmethod
    def forward(ctx, u, dt, a, b, c, d, z, dt_bias, h0, softplus, reset, lengths):
        y, h, saved = ssm.ssm_scan_fwd(u, dt, a, b, c, d, z, dt_bias, h0, softplus=softplus, reset=reset, lengths=lengths,
                                       want_saved=any(ctx.needs_input_grad))
        ctx.save_for_backward(u, dt, a, b, c, d, z, dt_bias, reset, lengths, saved)
        ctx.softplus, ctx.has_h0 = softplus, h0 is not None
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        u, dt, a, b, c, d, z, dt_bias, reset, lengths, saved = ctx.saved_tensors
        # expanded cotangents (of a sum) have no rows to read: lay them out
        dy = torch.zeros_like(u, memory_format=torch.contiguous_format) if dy is None else dy.contiguous()
        dh = None if dh is None else dh.contiguous()
        g = ssm.ssm_scan_bwd(u, dt, a, b, c, d, z, dt_bias, saved, dy, dh, softplus=ctx.softplus, reset=reset, lengths=lengths, want_dh0=ctx.has_h0)
        grads = tuple(g.get(k) for k in ("du", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dh0"))
        return (*_once("ssm_scan", grads, u, dt, a, b, c, d, z, dt_bias, dy, dh), None, None, None)


def ssm_scan(u, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, *, softplus=True, reset=None, lengths=None):
    """Selective state space scan with its gate; returns (y, h_final)."""
    return SsmScan.apply(u, dt, a, b, c, d, z, dt_bias, h0, softplus, reset, lengths)


class CausalConv(torch.autograd.Function):
    """Short causal convolution: (x, w, bias, state) -> (y, state_out), as
    ssm.causal_conv_fwd.  A second derivative raises."""

    @staticmethod
    def forward(ctx, x, w, bias, state, act, reset, lengths):
        y, last = ssm.causal_conv_fwd(x, w, bias, act=act, state=state, reset=reset, lengths=lengths)
        ctx.save_for_backward(x, w, bias, state, reset, lengths)
        ctx.act = act
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    def backward(ctx, dy, dlast):
        x, w, bias, state, reset, lengths = ctx.saved_tensors
        dy = torch.zeros_like(x, memory_format=torch.contiguous_format) if dy is None else dy.contiguous()
        dlast = None if dlast is None else dlast.contiguous()
        g = ssm.causal_conv_bwd(x, w, bias, dy, dlast, act=ctx.act, state=state, reset=reset, lengths=lengths)
        grads = tuple(g.get(k) for k in ("dx", "dw", "dbias", "dstate"))
        return (*_once("causal_conv", grads, x, w, bias, state, dy, dlast), None, None, None)


def causal_conv(x, w, bias=None, state=None, *, act="silu", reset=None, lengths=None):
    """Short causal convolution of each channel over time; returns (y, state_out)."""
    return CausalConv.apply(x, w, bias, state, act, reset, lengths)
