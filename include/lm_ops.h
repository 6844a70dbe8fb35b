/*
 * lm_ops.h -- C ABI of the language-model operators that stand around the
 * recurrent mixers of samu_scan.h on MI355X (gfx950): the norms before and
 * after a block with its gate and residual scale, the softmax cross entropy of
 * a linear head without the logits, and the AdamW step over many tensors.
 *
 * Conventions are those of samu_scan.h (device pointers, asynchronous on
 * `stream`, all arguments validated before the first enqueue, no allocation,
 * caller-owned buffers, gradients overwrite, bitwise deterministic, errors by
 * scan_status and scan_last_error()) with these differences:
 *   - activations are rows with a stride in elements between them (columns
 *     dense), so parts of a wider projection are taken as they lie;
 *   - norm and AdamW pointers need only the alignment of their element type.
 */
#ifndef LM_OPS_H
#define LM_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "samu_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ======================================================================
 * Block norms.  For each row, with x the residual stream, y the block's
 * output (the branch), g its gate logits:
 *   full form (w_post and scale given):
 *     rs1 = (mean(y^2) + eps)^-1/2,  u = scale * act(g) * (y rs1 w_post)
 *   plain form (both NULL):          u = act(g) * y
 *   r = x + u,  rs2 = (mean(r^2) + eps)^-1/2,  n = r rs2 w_pre.
 * act is 1 (LM_GATE_NONE, gate NULL), sigmoid(g) or g sigmoid(g) (SiLU).
 * Arithmetic is FP32; r (stream type) and n (branch type) are rounded once,
 * and n is formed from the unrounded r.
 * ====================================================================== */
enum { LM_GATE_NONE = 0, LM_GATE_SIGMOID = 1, LM_GATE_SILU = 2 };

/* Widest row of the block norms. */
#define LM_NORM_MAX_D 16384

/* Forward.
 *   x     [rows, d] of stream_dtype, row stride x_stride
 *   y     [rows, d] of branch_dtype; gate the same or NULL
 *   w_post, scale  f32 [d], both or neither;  w_pre  f32 [d]
 *   r     [rows, d] of stream_dtype, dense; may be x itself where x is dense
 *         (the backward reads x as it was before)
 *   n     [rows, d] of branch_dtype, dense
 *   stats f32 [rows, 2]: (rs1, rs2) for the backward (rs1 = 1 in the plain form)
 * rows >= 0 (0: nothing to do), 1 <= d <= LM_NORM_MAX_D. */
scan_status lm_block_norm_fwd(int64_t rows, int d, int stream_dtype, int branch_dtype, int gate_act, double eps,
                              const void* x, int64_t x_stride, const void* y, int64_t y_stride,
                              const void* gate, int64_t gate_stride,
                              const float* w_post, const float* scale, const float* w_pre,
                              void* r, void* n, float* stats, void* stream);

/* Backward for the cotangents dr (of r, stream type) and dn (of n, branch
 * type); either may be NULL (= 0).  With rh = r rs2, yh = y rs1, t = dn w_pre:
 *   dx = v = dr + rs2 (t - rh mean(t rh)),  dw_pre = sum dn rh,
 *   q = v scale act w_post,  dy = rs1 (q - yh mean(q yh))  (plain: dy = v act),
 *   dgate = v scale yh w_post act'(g),
 *   S = sum v act yh,  dw_post = scale S,  dscale = w_post S.
 *   dx stream type, dy and dgate branch type, dense; dgate NULL without a
 *   gate; dw_post, dscale f32 [d] (NULL in the plain form); dw_pre f32 [d].
 * Column sums are per-workgroup FP32 partials over fixed rows, then a
 * fixed-order FP64 sum.  rows = 0 zeroes the weight gradients.
 *   workspace  lm_block_norm_bwd_workspace_bytes(rows, d) bytes */
size_t lm_block_norm_bwd_workspace_bytes(int64_t rows, int d);
scan_status lm_block_norm_bwd(int64_t rows, int d, int stream_dtype, int branch_dtype, int gate_act,
                              const void* x, int64_t x_stride, const void* y, int64_t y_stride,
                              const void* gate, int64_t gate_stride,
                              const float* w_post, const float* scale, const float* w_pre,
                              const float* stats, const void* dr, int64_t dr_stride,
                              const void* dn, int64_t dn_stride,
                              void* dx, void* dy, void* dgate, float* dw_post, float* dscale, float* dw_pre,
                              void* workspace, size_t workspace_bytes, void* stream);

/* ======================================================================
 * Softmax cross entropy of a linear head, without the logits in memory.  For
 * token t with hidden row h_t, vocabulary rows w_j and target y_t:
 *   z_j = h_t . w_j   (softcap > 0: softcap tanh(h_t . w_j / softcap)),
 *   lse_t = log sum_j exp z_j,  loss_t = lse_t - z_{y_t}.
 * BF16 matrix-core products with FP32 sums.  A negative target: the token does
 * not count (loss 0, and dloss is not read for it; lse is formed all the
 * same).  A target >= v: loss and gradients are NaN.
 *   h       bf16 [n, d], row stride h_stride (a multiple of 8)
 *   w       bf16 [v, d]
 *   target  int64 [n]
 * 0 <= n <= 2^26 - 16, 1 <= v < 2^31 - 513, n v < 2^45; 8 <= d <= 65536, a multiple of 8;
 * n d <= 2^34 - 1024; h and w 16-byte aligned.  The backward works on the tokens with a weight alone
 * (dloss of a token that counts, or dlse, not zero): the others cost it nothing, and
 * whatever their hidden rows hold, NaN and infinities too, stays out of dw.
 * ====================================================================== */

/* Forward: loss, lse f32 [n].
 *   workspace  lm_linear_ce_workspace_bytes(n, d, v, 0) bytes */
size_t lm_linear_ce_workspace_bytes(int64_t n, int d, int64_t v, int backward);
scan_status lm_linear_ce_fwd(int64_t n, int d, int64_t v, double softcap, const void* h, int64_t h_stride,
                             const void* w, const int64_t* target, float* loss, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Backward for the cotangents dloss f32 [n] and dlse f32 [n] (NULL = 0), from
 * the forward's lse; the logits are formed again, some of the vocabulary at a
 * time:
 *   dz = (exp(z - lse) (dloss + dlse) - onehot(y) dloss) (1 - tanh^2),
 *   dh = dz w,  dw = dz^T h,
 * with dz rounded to BF16 for the two products, also where grad_dtype is FP32 (a
 * term is off by up to 2^-8 of itself).  dh [n, d] and dw [v, d] are of grad_dtype, dense.
 *   workspace  lm_linear_ce_workspace_bytes(n, d, v, 1) bytes */
scan_status lm_linear_ce_bwd(int64_t n, int d, int64_t v, double softcap, const void* h, int64_t h_stride,
                             const void* w, const int64_t* target, const float* lse, const float* dloss,
                             const float* dlse, void* dh, void* dw, int grad_dtype,
                             void* workspace, size_t workspace_bytes, void* stream);

/* ======================================================================
 * AdamW over many tensors, in place.  For every element, in FP32:
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   p = p (1 - lr decay) - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps).
 * p is read from `master` (FP32) where there is one, else from p itself, and
 * rounded to p's type once.
 *   state_bits 32: m, v are f32 [n].
 *   state_bits 8: m, v are e4m3 codes [n] with FP32 scales [ceil(n / 256)], one
 *     a block of 256 consecutive elements; v's codes hold sqrt(v).  A block's
 *     scale is max(|.|) / 448, at least 2^-96; a positive sqrt(v) takes at
 *     least the least positive code, so that no element's step is divided by
 *     eps alone.  A NaN in a block makes its scale NaN.
 * Arrays hold `count` entries (host memory, read before the call returns):
 * p, g, m, v, n (elements), decay; master (or NULL), m_scale, v_scale (8 bits).
 * All tensors of a call share their types; tensors may not overlap.
 * ====================================================================== */
#define LM_ADAMW_BLOCK 256
scan_status lm_adamw_step(int count, int param_dtype, int grad_dtype, int state_bits,
                          void* const* p, const void* const* g, void* const* m, void* const* v,
                          float* const* master, float* const* m_scale, float* const* v_scale,
                          const int64_t* n, const double* decay,
                          double lr, double beta1, double beta2, double eps, int64_t step, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LM_OPS_H */
