// lm_norm.hip -- the norms before and after a block, with its gate and
// residual scale, forward and backward.
//
// For a row of width d, with y the block's output, g its gate logits and x
// the residual stream (FP32 arithmetic; without w_post and scale the first
// norm and both weights are left out):
//   u = scale act(g) (y rs1) w_post,  r = x + u,  n = (r rs2) w_pre,
//   rs1 = (mean y^2 + eps)^-1/2,  rs2 = (mean r^2 + eps)^-1/2.
// Backward, from x, y, g and the kept (rs1, rs2) of each row:
//   t = dn w_pre, rh = r rs2, v = dr + rs2 (t - rh mean(t rh)), dx = v,
//   q = v scale act w_post, yh = y rs1, dy = rs1 (q - yh mean(q yh)),
//   dgate = v scale yh w_post act',
//   column sums: dw_pre = sum dn rh and S = sum v act yh, of which both
//   dw_post = scale S and dscale = w_post S follow.
//
// Bound by memory: each row is read once into registers, both reductions and
// every output come from there.  A row belongs to W waves of a workgroup, each
// lane holding NV groups of 4 consecutive elements, 256 W elements apart, so
// every load of a wave covers whole lines.  With W = 1 a workgroup holds four
// rows (eight or 16 of up to 128 or 64 columns, on half or a quarter of a wave) and needs no barrier.  Workgroups walk over rows with the weights in
// registers, and the backward keeps its column sums there until the end.
// 32768 x 2560, FP32 stream and BF16 branch with a gate, call after call: forward 217 us, 5.4 TB/s;
// backward 312 us with the column sums, 5.9 TB/s (a large copy runs at 4.8 TB/s; traced one by one the two take 222 and 342 us).
// Above 8192 columns the backward's four groups a lane do not fit the 128 registers of a 16-wave workgroup: 65 to 199 spill,
// and 4096 x 16384 BF16 takes 445 us, 2.4 TB/s (878 where the width is odd); the forward does not spill (147 us, 4.6 TB/s).
#include "lm.hpp"

namespace lrs {
namespace {

constexpr int MAX_WAVES = 16;

// Sum over the row's lanes: L, or (L = 0) the workgroup's.  `slot` alternates between calls, so one barrier
// a reduction is enough: a slot is written again only after the barrier of the
// reduction in between.
template <int L>
__device__ __forceinline__ float row_sum(float v, float (*slots)[MAX_WAVES], int slot, int waves) {
    if (L > 0 && L < 64) {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
        return v;
    }
    v = wave_sum(v);
    if (L > 0) return v;
    if ((threadIdx.x & 63) == 0) slots[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < waves; ++i) s += slots[slot][i];
    return s;
}

__device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}

// s = sigmoid(g) and 1 - s, which of a large g is far smaller than s's own rounding: with e = exp(-g), 1 - s = e s.  An e beyond
// 2^126, where s is less than FP32 holds, leaves 1.
__device__ __forceinline__ float sigmoid(float g, float* rest) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504f * g), s = __builtin_amdgcn_rcpf(1.0f + e);
    *rest = e > 0x1p126f ? 1.0f : e * s;
    return s;
}

// Which elements a lane holds: group c starts at column c * 4 T + 4 t.  Where
// the width is no multiple of 4 (TAIL) the group that the row ends in is loaded as the
// row's last four elements and put in place by take(), so that no load stands in a
// branch of its own (each would be waited for there).
template <class T, bool TAIL>
__device__ __forceinline__ Quad<T> row_load(const T* row, int col, int d) {
    if (TAIL) {
        if (d < 4) return col < d ? Quad<T>::load_some(row, d) : Quad<T>::zero();
        return Quad<T>::load(row + (col + 4 <= d ? col : d - 4));
    }
    if (col + 4 <= d) return Quad<T>::load(row + col);
    return Quad<T>::zero();
}
template <bool TAIL, class T>
__device__ __forceinline__ void take(const Quad<T>& q, int col, int d, float* f) {
    q.get(f);
    if (TAIL) {
        const int n = d < 4 && col < d ? 4 : d - col;  // this lane's elements, 4 or more: all
        if (n < 4) {
            const float a = f[1], b = f[2], c = f[3];
            f[0] = n == 3 ? a : n == 2 ? b : n == 1 ? c : 0.0f;
            f[1] = n == 3 ? b : n == 2 ? c : 0.0f;
            f[2] = n == 3 ? c : 0.0f;
            f[3] = 0.0f;
        }
    }
}
template <class T, bool TAIL>
__device__ __forceinline__ void row_store(T* row, int col, int d, const float* f) {
    if (col + 4 <= d) Quad<T>::store(row + col, f);
    else if (TAIL && col < d) Quad<T>::store_some(row + col, f, d - col);
}
template <bool TAIL>
__device__ __forceinline__ void weight_load(const float* w, int col, int d, float missing, float* f) {
    if (w) {
        take<TAIL>(row_load<float, TAIL>(w, col, d), col, d, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = missing;
    }
}

// TAIL: d is not a multiple of 4.  L: lanes of a row, 0: all of the workgroup's.
template <class ST, class BR, int NV, int L, bool TAIL>
__global__ __launch_bounds__(L > 0 ? 256 : 1024) void norm_fwd_kernel(const NormArgs a) {
    __shared__ float slots[2][MAX_WAVES];
    const int T = L > 0 ? L : blockDim.x, t = L > 0 ? threadIdx.x % L : threadIdx.x, waves = T >> 6;
    const int per = L > 0 ? 256 / L : 1, mine = L > 0 ? threadIdx.x / L : 0;
    const bool full = a.w_post != nullptr, gated = a.gate != nullptr, silu = a.gate_act == 2;
    const float inv_d = 1.0f / (float)a.d;
    float w1[NV][4], w2[NV][4];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int col = c * 4 * T + 4 * t;
        float sc[4];
        weight_load<TAIL>(a.w_post, col, a.d, 1.0f, w1[c]);
        weight_load<TAIL>(a.scale, col, a.d, 1.0f, sc);
        weight_load<TAIL>(a.w_pre, col, a.d, 1.0f, w2[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) w1[c][i] *= sc[i];  // scale and w_post act as one factor of u
    }
    for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < a.rows; row0 += (int64_t)gridDim.x * per) {
        const int64_t row = row0 + mine;
        if (L > 0 && row >= a.rows) break;  // no barrier in this form
        Quad<ST> qx[NV];
        Quad<BR> qy[NV], qg[NV];
        const ST* x = static_cast<const ST*>(a.x) + row * a.x_stride;
        const BR* y = static_cast<const BR*>(a.y) + row * a.y_stride;
        const BR* g = static_cast<const BR*>(a.gate) + row * a.gate_stride;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = c * 4 * T + 4 * t;
            qy[c] = row_load<BR, TAIL>(y, col, a.d);
            if (gated) qg[c] = row_load<BR, TAIL>(g, col, a.d);
            qx[c] = row_load<ST, TAIL>(x, col, a.d);
        }
        float rs1 = 1.0f;
        if (full) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                float f[4];
                take<TAIL>(qy[c], c * 4 * T + 4 * t, a.d, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) s = fmaf(f[i], f[i], s);
            }
            rs1 = 1.0f / sqrtf(row_sum<L>(s, slots, 0, waves) * inv_d + a.eps);
        }
        float r[NV][4], s = 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            float f[4], u[4];
            take<TAIL>(qy[c], c * 4 * T + 4 * t, a.d, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = u[i] * rs1 * w1[c][i];
            if (gated) {
                take<TAIL>(qg[c], c * 4 * T + 4 * t, a.d, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float sg = sigmoid(f[i]);
                    u[i] *= silu ? sg * f[i] : sg;
                }
            }
            take<TAIL>(qx[c], c * 4 * T + 4 * t, a.d, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[c][i] = f[i] + u[i];
                s = fmaf(r[c][i], r[c][i], s);
            }
        }
        const float rs2 = 1.0f / sqrtf(row_sum<L>(s, slots, 1, waves) * inv_d + a.eps);
        ST* ro = static_cast<ST*>(a.r) + row * a.d;
        BR* no = static_cast<BR*>(a.n) + row * a.d;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = c * 4 * T + 4 * t;
            row_store<ST, TAIL>(ro, col, a.d, r[c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) r[c][i] = r[c][i] * rs2 * w2[c][i];
            row_store<BR, TAIL>(no, col, a.d, r[c]);
        }
        if (t == 0) {
            a.stats[2 * row] = rs1;
            a.stats[2 * row + 1] = rs2;
        }
        // the plain form has one reduction a row: keep its slot from being written while others still read it
        if (L == 0 && !full) __syncthreads();
    }
}

template <class ST, class BR, int NV, int L, bool TAIL>
__global__ __launch_bounds__(L > 0 ? 256 : 1024) void norm_bwd_kernel(const NormArgs a) {
    __shared__ float slots[2][MAX_WAVES];
    const int T = L > 0 ? L : blockDim.x, t = L > 0 ? threadIdx.x % L : threadIdx.x, waves = T >> 6;
    const int per = L > 0 ? 256 / L : 1, mine = L > 0 ? threadIdx.x / L : 0;
    const bool full = a.w_post != nullptr, gated = a.gate != nullptr, silu = a.gate_act == 2;
    const float inv_d = 1.0f / (float)a.d;
    float w1[NV][4], w2[NV][4], sum2[NV][4], sums[NV][4];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int col = c * 4 * T + 4 * t;
        float sc[4];
        weight_load<TAIL>(a.w_post, col, a.d, 1.0f, w1[c]);
        weight_load<TAIL>(a.scale, col, a.d, 1.0f, sc);
        weight_load<TAIL>(a.w_pre, col, a.d, 1.0f, w2[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w1[c][i] *= sc[i];
            sum2[c][i] = sums[c][i] = 0.0f;
        }
    }
    for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < a.rows; row0 += (int64_t)gridDim.x * per) {
        const int64_t row = row0 + mine;
        if (L > 0 && row >= a.rows) break;
        Quad<ST> qx[NV], qr[NV];
        Quad<BR> qy[NV], qg[NV], qn[NV];
        const ST* x = static_cast<const ST*>(a.x) + row * a.x_stride;
        const BR* y = static_cast<const BR*>(a.y) + row * a.y_stride;
        const BR* g = static_cast<const BR*>(a.gate) + row * a.gate_stride;
        const ST* dr = static_cast<const ST*>(a.dr) + row * a.dr_stride;
        const BR* dn = static_cast<const BR*>(a.dn) + row * a.dn_stride;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = c * 4 * T + 4 * t;
            qy[c] = row_load<BR, TAIL>(y, col, a.d);
            if (gated) qg[c] = row_load<BR, TAIL>(g, col, a.d);
            qx[c] = row_load<ST, TAIL>(x, col, a.d);
            qn[c] = a.dn ? row_load<BR, TAIL>(dn, col, a.d) : Quad<BR>::zero();
            qr[c] = a.dr ? row_load<ST, TAIL>(dr, col, a.d) : Quad<ST>::zero();
        }
        const float rs1 = a.stats[2 * row], rs2 = a.stats[2 * row + 1];
        // rh = r rs2 and the first mean, of t rh; act(g) and yh are formed
        // again where they are used, which costs less than keeping them
        float rh[NV][4], s = 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            float u[4], f[4];
            take<TAIL>(qy[c], c * 4 * T + 4 * t, a.d, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = u[i] * rs1 * w1[c][i];
            if (gated) {
                take<TAIL>(qg[c], c * 4 * T + 4 * t, a.d, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float sg = sigmoid(f[i]);
                    u[i] *= silu ? sg * f[i] : sg;
                }
            }
            take<TAIL>(qx[c], c * 4 * T + 4 * t, a.d, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) rh[c][i] = (f[i] + u[i]) * rs2;
            take<TAIL>(qn[c], c * 4 * T + 4 * t, a.d, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = f[i] * rh[c][i];
                sum2[c][i] += p;
                s = fmaf(p, w2[c][i], s);
            }
        }
        const float m2 = row_sum<L>(s, slots, 0, waves) * inv_d;
        // v, dx, dgate, the column sum S, and q yh for the second mean
        ST* dx = static_cast<ST*>(a.dx) + row * a.d;
        BR* dy = static_cast<BR*>(a.dy) + row * a.d;
        BR* dg = static_cast<BR*>(a.dgate) + row * a.d;
        s = 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = c * 4 * T + 4 * t;
            float v[4], f[4], yh[4], da[4];
            take<TAIL>(qr[c], c * 4 * T + 4 * t, a.d, v);
            take<TAIL>(qn[c], c * 4 * T + 4 * t, a.d, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += rs2 * (f[i] * w2[c][i] - rh[c][i] * m2);
            row_store<ST, TAIL>(dx, col, a.d, v);
            take<TAIL>(qy[c], c * 4 * T + 4 * t, a.d, yh);
#pragma unroll
            for (int i = 0; i < 4; ++i) yh[i] *= rs1;
            if (gated) {
                take<TAIL>(qg[c], c * 4 * T + 4 * t, a.d, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float rest;
                    const float sg = sigmoid(f[i], &rest), slope = sg * rest;
                    da[i] = v[i] * yh[i] * w1[c][i] * (silu ? sg + f[i] * slope : slope);
                    v[i] *= silu ? sg * f[i] : sg;
                }
                row_store<BR, TAIL>(dg, col, a.d, da);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sums[c][i] += v[i] * yh[i];
                rh[c][i] = v[i] * w1[c][i];  // q
                s = fmaf(rh[c][i], yh[i], s);
            }
        }
        const float m1 = full ? row_sum<L>(s, slots, 1, waves) * inv_d : 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = c * 4 * T + 4 * t;
            float yh[4];
            take<TAIL>(qy[c], c * 4 * T + 4 * t, a.d, yh);
            if (full) {
#pragma unroll
                for (int i = 0; i < 4; ++i) rh[c][i] = rs1 * (rh[c][i] - yh[i] * rs1 * m1);
            }
            row_store<BR, TAIL>(dy, col, a.d, rh[c]);
        }
        if (L == 0 && !full) __syncthreads();
    }
    // column sums of this workgroup's rows (in a fixed order over its waves)
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.d;
    if (L > 0) {
        constexpr int ROWS = L > 0 ? 256 / L : 1, LINE = NV * 4 * (L > 0 ? L : 1);
        __shared__ float buf[ROWS][LINE];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k) __syncthreads();
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) buf[mine][c * 4 * L + 4 * t + i] = k ? sums[c][i] : sum2[c][i];
            __syncthreads();
            for (int col = threadIdx.x; col < a.d; col += 256) {
                float s = 0.0f;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) s += buf[r][col];
                part[k * a.d + col] = s;
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = c * 4 * T + 4 * t + i;
                if (col < a.d) {
                    part[col] = sum2[c][i];
                    part[a.d + col] = sums[c][i];
                }
            }
    }
}

// Column sums over the workgroups' partials, FP64 in a fixed order: 16
// columns a workgroup, 64 lanes down each column, eight loads of a lane at a
// time.  blockIdx.y: dw_pre, or S and from it dw_post and dscale.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* part, int blocks, int d, const float* w_post,
                                                           const float* scale, float* dw_post, float* dscale,
                                                           float* dw_pre) {
    __shared__ double buf[16][17];
    const int c = threadIdx.x & 15, lane = threadIdx.x >> 4, col = blockIdx.x * 16 + c, k = blockIdx.y;
    double s = 0.0;
    if (col < d)
        for (int i = lane; i < blocks; i += 64 * 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = i + 64 * u < blocks ? part[((int64_t)(i + 64 * u) * 2 + k) * d + col] : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) s += (double)v[u];
        }
    // four of a wave's lanes share a column, then the 16 waves do
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if ((lane & 3) == 0) buf[lane >> 2][c] = s;
    __syncthreads();
    if (lane == 0 && col < d) {
        double v = buf[0][c];
#pragma unroll
        for (int i = 1; i < 16; ++i) v += buf[i][c];
        if (k == 0) {
            dw_pre[col] = (float)v;
        } else {
            dw_post[col] = (float)(v * (double)scale[col]);
            dscale[col] = (float)(v * (double)w_post[col]);
        }
    }
}

// Waves of a row: NV groups of 256 columns a wave.  Times are of BF16 calls, column sums included; one plan serves both
// directions, whose rows lie alike.
//   Few rows leave the chip idle however they are spread, so they take one group a lane (the shortest
// chain of loads and sums).  The backward of 512 x 4096: 19.9 us, 24.5 with two groups; of 512 x 2048 16.5 and 17.0; of 1024 x 1024
// 13.6 and 12.5, of 1024 x 512 13.8 and 11.8 (1024 x 2048 would still gain, 19.3 and 20.5).  The forward of so few is a launch either way, 6 us.
//   Of many rows, those up to 1024 columns are one wave's: four rows are then in flight in a workgroup and no barrier stands
// between them.  Backward of 4096 x 1024 22.8 us, 29.0 with two waves a row; of 32768 x 1024 102.6 and 111.3.  Forward of the two 10.9 and 9.9,
// 63.0 and 62.8.  Up to 128 and 64 columns half a wave's or a quarter's: 32768 x 64 backward 14 us, 32 with a wave a row, forward 7.6 and 15.1;
// 32768 x 128 backward 21.7 and 28.4, forward 12.4 and 16.7.
//   Wider ones take two groups a wave, four above 8192
// columns, where a row would not fit the 16 waves of a workgroup.
struct Plan {
    int nv, waves, lanes;  // lanes of a row where it is no more than a wave's, else 0
};
Plan plan(int64_t rows, int d) {
    const int groups = (int)ceil_div(d, 256);
    if (groups == 1) return {1, 1, d <= 64 ? 16 : d <= 128 ? 32 : 64};
    if (rows <= 512 && groups <= MAX_WAVES) return {1, groups, 0};
    if (groups > 2 && groups <= 4) return {4, 1, 64};
    if (groups <= 2 * MAX_WAVES) return {2, (int)ceil_div(groups, 2), groups <= 2 ? 64 : 0};
    return {4, (int)ceil_div(groups, 4), 0};
}

template <bool BWD, class ST, class BR, int NV, int L>
void launch_one(const NormArgs& a, dim3 g, dim3 b, hipStream_t s) {
    if (a.d % 4 == 0) {
        if (BWD) LRS_LAUNCH(K_LM_NORM_BWD, (norm_bwd_kernel<ST, BR, NV, L, false>), g, b, 0, s, a);
        else LRS_LAUNCH(K_LM_NORM, (norm_fwd_kernel<ST, BR, NV, L, false>), g, b, 0, s, a);
    } else {
        if (BWD) LRS_LAUNCH(K_LM_NORM_BWD, (norm_bwd_kernel<ST, BR, NV, L, true>), g, b, 0, s, a);
        else LRS_LAUNCH(K_LM_NORM, (norm_fwd_kernel<ST, BR, NV, L, true>), g, b, 0, s, a);
    }
}

template <bool BWD, class ST, class BR>
void launch_typed(const NormArgs& a, int blocks, hipStream_t s) {
    const Plan p = plan(a.rows, a.d);
    const dim3 g(blocks), b(p.lanes ? 256 : 64 * p.waves);
    if (p.lanes) {
        if (p.lanes == 16) launch_one<BWD, ST, BR, 1, 16>(a, g, b, s);
        else if (p.lanes == 32) launch_one<BWD, ST, BR, 1, 32>(a, g, b, s);
        else if (p.nv == 1) launch_one<BWD, ST, BR, 1, 64>(a, g, b, s);
        else if (p.nv == 2) launch_one<BWD, ST, BR, 2, 64>(a, g, b, s);
        else launch_one<BWD, ST, BR, 4, 64>(a, g, b, s);
    } else {
        if (p.nv == 1) launch_one<BWD, ST, BR, 1, 0>(a, g, b, s);
        else if (p.nv == 2) launch_one<BWD, ST, BR, 2, 0>(a, g, b, s);
        else launch_one<BWD, ST, BR, 4, 0>(a, g, b, s);
    }
}

template <bool BWD>
void launch_any(const NormArgs& a, int stream_f32, int branch_f32, int blocks, hipStream_t s) {
    if (stream_f32) {
        if (branch_f32) launch_typed<BWD, float, float>(a, blocks, s);
        else launch_typed<BWD, float, uint16_t>(a, blocks, s);
    } else {
        if (branch_f32) launch_typed<BWD, uint16_t, float>(a, blocks, s);
        else launch_typed<BWD, uint16_t, uint16_t>(a, blocks, s);
    }
}

}  // namespace

// Workgroups that walk over the rows.  Each writes its column sums, and HBM
// serves few long streams better than many.  Half of them, these, 1.5 and 2 times as many take, in BF16 but for the first:
//   5 waves a row   32768 x 2560, FP32 stream   484, 312, 378, 410 us
//   16              4096 x 8192                 186, 130, 157, 142
//   3               8192 x 1536                  59,  52,  62,  61
//   one             32768 x 1024                126, 103, 115, 109
//   one, narrow     32768 x 256                  39,  33,  37,  43
//   half, a quarter 32768 x 128, x 64            23,  21,  24,  28;  19, 14, 15, 16
int lm_norm_bwd_blocks(int64_t rows, int d) {
    const Plan p = plan(rows, d);
    const int most = p.lanes ? (d > 64 && d <= 256 ? 1024 : 512) : p.waves > 8 ? 256 : p.waves >= 4 ? 512 : 1024;
    return (int)std::min<int64_t>(ceil_div(rows, p.lanes ? 256 / p.lanes : 1), most);
}

// The forward keeps nothing between rows, and its count matters little: with more than 8 waves a row 768 workgroups take
// 70 us for 4096 x 8192, 4096 72; with fewer waves 4096 take 82 us for 32768 x 1280 and 217 for 32768 x 2560 with an FP32 stream, 768 102 and 213.
hipError_t launch_norm_fwd(const NormArgs& a, int stream_f32, int branch_f32, hipStream_t s) {
    const Plan p = plan(a.rows, a.d);
    launch_any<false>(a, stream_f32, branch_f32,
                      (int)std::min<int64_t>(ceil_div(a.rows, p.lanes ? 256 / p.lanes : 1), p.waves > 8 ? 768 : 4096), s);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, int stream_f32, int branch_f32, float* dw_post, float* dscale,
                           float* dw_pre, hipStream_t s) {
    const int blocks = a.rows ? lm_norm_bwd_blocks(a.rows, a.d) : 0;
    if (blocks) launch_any<true>(a, stream_f32, branch_f32, blocks, s);
    LRS_LAUNCH(K_LM_NORM_REDUCE, norm_reduce_kernel, dim3((unsigned)ceil_div(a.d, 16), a.w_post ? 2 : 1), dim3(1024), 0, s,
               (const float*)a.part, blocks, a.d, a.w_post, a.scale, dw_post, dscale, dw_pre);
    return hipGetLastError();
}

}  // namespace lrs
