/*
 * ssm_ops.h -- C ABI of the selective state space mixer on MI355X (gfx950):
 * the scan with its gate, forward, backward and for single tokens, and the
 * short causal convolution in front of it.
 *
 * Conventions are those of samu_scan.h (device pointers, asynchronous on
 * `stream`, all arguments validated before the first enqueue, no allocation,
 * caller-owned buffers, gradients overwrite, bitwise deterministic, errors by
 * scan_status and scan_last_error()) with these differences:
 *   - rows of activations lie at a distance given in elements (columns dense),
 *     so parts of a wider projection are taken as they lie; row (i, t) of a
 *     [batch, length, ...] tensor is number i * length + t;
 *   - pointers need only the alignment of their element type.
 *
 * Rows of several sequences.  `reset` uint8 [batch, length] (NULL: none): a
 * token with a flag starts a sequence, and nothing from before reaches it, no
 * NaN either.  `lengths` int32 [batch] (NULL: all of `length`): tokens from
 * there on are padding: their outputs and gradients are zero, what their
 * inputs hold is not used, and the state behind a row is the one after its
 * last token.  A length outside 0..length counts as the nearest of the two.
 * The two operators differ on flags in the padding: for the scan one starts an empty
 * sequence there, whose state behind the row is then zero; the convolution looks at no
 * flags there and leaves the inputs of the row's last tokens.  Where single tokens go on
 * from both states, clear the flags of padding first (reset and t < lengths).
 */
#ifndef SSM_OPS_H
#define SSM_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "samu_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ======================================================================
 * Selective scan.  For token t, channel i (of group k = i / (d / groups)) and
 * state j:
 *   x_t = dt_t + dt_bias,  s_t = softplus(x_t)  (softplus = 0: x_t),
 *   h_t = exp(s_t a) h_{t-1} + s_t u_t b_t,
 *   y_t = (sum_j c_t h_t + d u_t) z_t sigmoid(z_t)     (z NULL: no gate).
 * Arithmetic and states are FP32; y is rounded once.
 *   u, dt, z  [batch, length, d] of dtype;  b, c  [batch, length, groups, n] of
 *   dtype, a row's groups * n values dense;  a f32 [d, n];  skip (d above) and
 *   dt_bias f32 [d], NULL = 0;  h0 f32 [batch, d, n], NULL = 0.
 * batch, length >= 0, 1 <= d <= 2^21 and a multiple of groups, 1 <= n <= SSM_MAX_STATE,
 * batch * length < 2^31, row strides below 2^22 (of a single token: up to 2^40), and fewer than
 * 2^24 waves: batch * groups * ceil((d / groups) / (128 / g)), g = 2, 4, 8, 16 for n up to 8, 16, 32, 64.
 * ====================================================================== */
#define SSM_MAX_STATE 64
/* Tokens between two states that the forward keeps for the backward. */
#define SSM_CHUNK 16

/* Forward.
 *   y        [batch, length, d] of dtype, dense
 *   h_final  f32 [batch, d, n]
 *   saved    ssm_scan_saved_bytes() bytes for the backward, or NULL: nothing is kept
 *   workspace  ssm_scan_workspace_bytes(..., 0) bytes
 * Sizes of 0 bytes mean an unsupported shape. */
size_t ssm_scan_saved_bytes(int64_t batch, int64_t length, int d, int n, int groups);
size_t ssm_scan_workspace_bytes(int64_t batch, int64_t length, int d, int n, int groups, int backward);
scan_status ssm_scan_fwd(int64_t batch, int64_t length, int d, int n, int groups, int dtype, int softplus,
                         const void* u, int64_t u_stride, const void* dt, int64_t dt_stride, const float* a,
                         const void* b, int64_t b_stride, const void* c, int64_t c_stride, const float* skip,
                         const void* z, int64_t z_stride, const float* dt_bias, const float* h0,
                         const uint8_t* reset, const int32_t* lengths, void* y, float* h_final, void* saved,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Backward for the cotangents dy [batch, length, d] of dtype and dh_final f32
 * [batch, d, n] (NULL = 0), from the forward's inputs and saved states.  With
 * e_t = dy_t z_t sigmoid(z_t), g_t = c_t e_t + exp(s_{t+1} a) g_{t+1}, r_t = exp(s_t a) g_t h_{t-1}:
 *   du = s sum_j g b + d e,  ds = u sum_j g b + sum_j a r,  ddt = ds softplus'(x),
 *   dc = sum_i e h,  db = sum_i s u g,  da = sum_t s r,  dskip = sum_t e u,
 *   ddt_bias = sum_t ddt,  dz = dy (sum_j c h + d u) (z sigmoid(z))',  dh0 = exp(s_0 a) g_0.
 * All are dense: du, ddt, dz [batch, length, d] and db, dc [batch, length, groups, n] of
 * dtype, da f32 [d, n], dskip and ddt_bias f32 [d], dh0 f32 [batch, d, n].
 * dskip, ddt_bias and dh0 may be NULL (not wanted); dz is NULL where z is.
 *   workspace  ssm_scan_workspace_bytes(..., 1) bytes */
scan_status ssm_scan_bwd(int64_t batch, int64_t length, int d, int n, int groups, int dtype, int softplus,
                         const void* u, int64_t u_stride, const void* dt, int64_t dt_stride, const float* a,
                         const void* b, int64_t b_stride, const void* c, int64_t c_stride, const float* skip,
                         const void* z, int64_t z_stride, const float* dt_bias, const uint8_t* reset,
                         const int32_t* lengths, const void* saved, const void* dy, int64_t dy_stride,
                         const float* dh_final, void* du, void* ddt, float* da, void* db, void* dc, float* dskip,
                         void* dz, float* ddt_bias, float* dh0, void* workspace, size_t workspace_bytes, void* stream);

/* One token of `batch` sequences: h f32 [batch, d, n], dense, is updated in place, y
 * [batch, d] of dtype, dense; the other tensors as above with length 1, row strides up to 2^40 (a
 * token's slice of longer rows). */
scan_status ssm_scan_step(int64_t batch, int d, int n, int groups, int dtype, int softplus, float* h, const void* u,
                          int64_t u_stride, const void* dt, int64_t dt_stride, const float* a, const void* b,
                          int64_t b_stride, const void* c, int64_t c_stride, const float* skip, const void* z,
                          int64_t z_stride, const float* dt_bias, void* y, void* stream);

/* ======================================================================
 * Short causal convolution of each channel over time, width 2 to
 * CONV_MAX_WIDTH:
 *   p_t = bias + sum_{j < width} w[width - 1 - j] x_{t-j},  y = act(p),
 * act CONV_NONE or CONV_SILU (p sigmoid(p)).  Inputs from before the row's
 * first token are the state's (state NULL: zero), inputs of an earlier
 * sequence of the row count as zero.  Arithmetic is FP32, y is rounded once.
 *   x      [batch, length, d] of dtype;  w f32 [d, width];  bias f32 [d], NULL = 0
 *   state  [batch, width - 1, d] of dtype, dense, the oldest input first
 * batch, length >= 0, 1 <= d <= 2^24, batch * length < 2^31, and launches below 2^32
 * threads: batch * pieces * ceil(d / 2) of pieces of 8 to 64 tokens.
 * ====================================================================== */
enum { CONV_NONE = 0, CONV_SILU = 1 };
#define CONV_MAX_WIDTH 4

/* Forward.  y [batch, length, d], dense.  state_out [batch, width - 1, d],
 * dense (NULL: not wanted): the inputs that the next token needs, zero where they are of an
 * earlier sequence; it may not be `state` itself. */
scan_status ssm_conv_fwd(int64_t batch, int64_t length, int d, int width, int dtype, int act, const void* x,
                         int64_t x_stride, const float* w, const float* bias, const void* state,
                         const uint8_t* reset, const int32_t* lengths, void* y, void* state_out, void* stream);

/* Backward for the cotangents dy (of y) and dstate_out (of state_out; NULL = 0).
 * With g = dy act'(p):
 *   dx_t = sum_j w[width - 1 - j] g_{t+j},  dw[width - 1 - j] = sum_t g_t x_{t-j},  dbias = sum_t g_t.
 *   dx [batch, length, d] and dstate [batch, width - 1, d] (NULL: not wanted)
 *   of dtype, dense; dw f32 [d, width]; dbias f32 [d] (NULL: not wanted).
 *   workspace  ssm_conv_bwd_workspace_bytes() bytes */
size_t ssm_conv_bwd_workspace_bytes(int64_t batch, int64_t length, int d, int width);
scan_status ssm_conv_bwd(int64_t batch, int64_t length, int d, int width, int dtype, int act, const void* x,
                         int64_t x_stride, const float* w, const float* bias, const void* state,
                         const uint8_t* reset, const int32_t* lengths, const void* dy, int64_t dy_stride,
                         const void* dstate_out, void* dx, float* dw, float* dbias, void* dstate, void* workspace,
                         size_t workspace_bytes, void* stream);

/* One token of `batch` sequences: x [batch, d], y [batch, d] (dense); state
 * [batch, width - 1, d] moves on by one input, in place. */
scan_status ssm_conv_step(int64_t batch, int d, int width, int dtype, int act, const void* x, int64_t x_stride,
                          const float* w, const float* bias, void* state, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_OPS_H */
