// lm_ce.hip -- softmax cross entropy of a linear head, forward and backward,
// without the logits in memory.
//
// For token t with hidden row h_t, vocabulary rows w_j and target y_t:
//   z_j = h_t . w_j, or c tanh(h_t . w_j / c) where logits are capped,
//   lse_t = log sum_j exp z_j,  loss_t = lse_t - z_{y_t} (0 where y_t < 0).
// The forward product's tiles end in a running maximum and sum of each token
// over the tile's vocabulary entries; a second small launch joins them.
// Backward, vocabulary chunk by chunk: the logits are formed again, and
//   dz_j = (exp(z_j - lse_t) (dloss_t + dlse_t) - [j = y_t] dloss_t) (1 - tanh^2)
// is rounded to BF16 (the operand type of the matrix cores; the error of a
// term is 2^-9 of it and independent from term to term) into a buffer of one
// chunk, from which both products follow,
//   dh += dz w_chunk (FP32 sums kept over the chunks),  dw_chunk = dz^T h.
//
// Bound by the matrix cores for many tokens (2 n d v flops forward, 6 n d v
// backward); by reading w for few.
#include "lm_gemm.hpp"

namespace lrs {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// Which tile a workgroup takes.  Workgroups go to the 8 XCDs in turn, so each
// XCD is given a contiguous run of tiles, and a run walks over groups of 8
// tiles along q for each tile along p: what 32 neighbouring tiles read stays in
// the XCD's L2.
__device__ __forceinline__ void tile_of(int np, int nq, int* p, int* q) {
    const int total = np * nq, b = blockIdx.x % total, xcd = b & 7, each = total >> 3, rest = total & 7;
    const int i = xcd * each + (xcd < rest ? xcd : rest) + (b >> 3);
    const int group = i / (8 * np), first = group * 8, size = nq - first < 8 ? nq - first : 8, in = i - first * np;
    *q = first + in % size;
    *p = in / size;
}

__device__ __forceinline__ float cap_tanh(float z, float inv_cap) {  // tanh(z / cap)
    return 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(2.0f * LOG2E * inv_cap * z));
}

// ------------------------------------------------------------- forward ---
// P = w (vocabulary), Q = h (tokens): a lane's results are 4 FM logits of each
// of FN tokens, so a token's maximum and sum are formed in registers and
// joined over the four lanes that share its column.
template <class T>
__global__ __launch_bounds__(T::THREADS) void ce_stats_kernel(const CeArgs a, int np, int nq) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tp, tq;
    tile_of(np, nq, &tp, &tq);
    constexpr int BM = T::P_BYTES / 128, BN = T::Q_BYTES / 128, WM = BM / 16 / T::FM;
    T t;
    t.run(lds, Operand{a.w, a.d, a.v}, Operand{a.h, a.h_stride, a.n}, tp * BM, tq * BN, 0, a.d);
    const int lane = threadIdx.x & 63;
    const int v0 = tp * BM + T::wave_p() + 4 * (lane >> 4), t0 = tq * BN + T::wave_q() + (lane & 15);
    const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int tok = t0 + 16 * j;
        const int64_t y = tok < a.n ? a.target[tok] : -1;
        float top = -__builtin_inff(), hit = 0.0f;
        bool mine = false;
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int v = v0 + 16 * i + r;
                float z = t.acc[i][j][r];
                if (a.cap > 0.0f) z = a.cap * cap_tanh(z, inv_cap);
                if (v == y && v < a.v) hit = z, mine = true;
                z = v < a.v ? z * LOG2E : -__builtin_inff();
                t.acc[i][j][r] = z;
                top = fmaxf(top, z);
            }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // an infinite maximum is not subtracted: inf - inf would be NaN where the sum is inf or 0
        const float base = fabsf(top) == __builtin_inff() ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) sum += __builtin_amdgcn_exp2f(t.acc[i][j][r] - base);
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (tok < a.n) {
            if (mine) a.picked[tok] = hit;
            if (lane < 16) {
                const int part = tp * WM + T::wave_p() / (BM / WM);
                reinterpret_cast<float2*>(a.part)[(int64_t)part * a.n + tok] = make_float2(top, sum);
            }
        }
    }
}

// Joins the partial maxima and sums of each token: 16 tokens a workgroup, 64 lanes each.
__global__ __launch_bounds__(1024) void ce_join_kernel(const CeArgs a, int parts) {
    __shared__ float2 buf[64][17];
    const int c = threadIdx.x & 15, l = threadIdx.x >> 4, tok = blockIdx.x * 16 + c;
    float top = -__builtin_inff(), sum = 0.0f;
    auto join = [&](float2 o) {
        const float m = fmaxf(top, o.x), base = fabsf(m) == __builtin_inff() ? 0.0f : m;
        sum = sum * __builtin_amdgcn_exp2f(top - base) + o.y * __builtin_amdgcn_exp2f(o.x - base);
        top = m;
    };
    if (tok < a.n)
        for (int i = l; i < parts; i += 64) join(reinterpret_cast<const float2*>(a.part)[(int64_t)i * a.n + tok]);
    buf[l][c] = make_float2(top, sum);
    __syncthreads();
    for (int o = 32; o > 0; o >>= 1) {
        if (l < o) {
            join(buf[l + o][c]);
            buf[l][c] = make_float2(top, sum);
        }
        __syncthreads();
    }
    if (l == 0 && tok < a.n) {
        const float base = fabsf(top) == __builtin_inff() ? 0.0f : top;
        const float lse = LN2 * (base + __builtin_amdgcn_logf(sum));
        const int64_t y = a.target[tok];
        a.lse[tok] = lse;
        // a target beyond the vocabulary has no loss: NaN says so
        a.loss[tok] = y < 0 ? 0.0f : y < a.v ? lse - a.picked[tok] : __builtin_nanf("");
    }
}

// ------------------------------------------------------------ backward ---
// The scale dz is held at: the largest |dloss| or |dloss + dlse| of a counting
// token.  BF16 rounds dloss itself, and where all tokens weigh the same it
// would round each target's entry the same way, an error that no sum averages
// out; over the scale, those entries are 1 - p.  Both products give it back.
__global__ __launch_bounds__(1024) void ce_scale_kernel(const CeArgs a) {
    __shared__ float buf[16];
    float top = 0.0f;
    for (int i = threadIdx.x; i < a.n; i += 1024) {
        const float dl = a.target[i] < 0 ? 0.0f : fabsf(a.dloss[i]);
        const float c = a.dlse ? fmaxf(dl, fabsf((a.target[i] < 0 ? 0.0f : a.dloss[i]) + a.dlse[i])) : dl;
        if (c < 0x1p100f) top = fmaxf(top, c);  // a weight that is not finite stays with its token
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i) top = fmaxf(top, buf[i]);
        *a.scale = top < 0x1p-100f ? 1.0f : top;
    }
}

// dz / scale of vocabulary entries [vfirst, vfirst + count), BF16 [n, ld]; columns from count
// to the next multiple of 64 are zeros.
template <class T>
__global__ __launch_bounds__(T::THREADS) void ce_dz_kernel(const CeArgs a, int np, int nq, int vfirst, int count, int ld) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tp, tq;
    tile_of(np, nq, &tp, &tq);
    constexpr int BM = T::P_BYTES / 128, BN = T::Q_BYTES / 128;
    T t;
    t.run(lds, Operand{static_cast<const char*>(a.w) + (int64_t)vfirst * a.d * 2, a.d, count}, Operand{a.h, a.h_stride, a.n},
          tp * BM, tq * BN, 0, a.d);
    const int lane = threadIdx.x & 63;
    const int v0 = tp * BM + T::wave_p() + 4 * (lane >> 4), t0 = tq * BN + T::wave_q() + (lane & 15);
    const int padded = (count + 63) / 64 * 64;
    const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f, inv_scale = 1.0f / *a.scale;
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int tok = t0 + 16 * j;
        if (tok >= a.n) continue;
        const int64_t y = a.target[tok];
        float dl = y < 0 ? 0.0f : a.dloss[tok];
        if (y >= a.v) dl = __builtin_nanf("");
        const float c = (dl + (a.dlse ? a.dlse[tok] : 0.0f)) * inv_scale, base = a.lse_in[tok] * LOG2E;
        dl *= inv_scale;
        const int64_t at = y - vfirst;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            float g[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int v = v0 + 16 * i + r;
                float z = t.acc[i][j][r], slope = 1.0f;
                if (a.cap > 0.0f) {
                    const float th = cap_tanh(z, inv_cap);
                    z = a.cap * th;
                    slope = (1.0f - th) * (1.0f + th);
                }
                // a token that takes no part gives exact zeros, whatever its logits are
                float x = c == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(fmaf(z, LOG2E, -base)) * c;
                if (v == at) x -= dl;
                g[r] = v < count ? x * slope : 0.0f;
            }
            const int v = v0 + 16 * i;
            if (v < padded) {
                uint16_t* o = static_cast<uint16_t*>(a.dz) + (int64_t)tok * ld + v;
                *reinterpret_cast<u32x2_t*>(o) = u32x2_t{pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3])};
            }
        }
    }
}

// dh_part[s] (+)= dz w_chunk over range s of the chunk.  P = w (width; the
// reduction index is not the dense one), Q = dz.
template <class T>
__global__ __launch_bounds__(T::THREADS) void ce_dh_kernel(const CeArgs a, int np, int nq, int vfirst, int count, int ld,
                                                           int range, int first) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tp, tq;
    tile_of(np, nq, &tp, &tq);
    constexpr int BM = T::P_BYTES / 128, BN = T::Q_BYTES / 128;
    const int split = blockIdx.x / (np * nq), k0 = split * range, k1 = k0 + range < count ? k0 + range : count;
    float* out = a.dh_part + (int64_t)split * a.n * a.d;
    T t;
    t.run(lds, Operand{static_cast<const char*>(a.w) + (int64_t)vfirst * a.d * 2, a.d, a.d}, Operand{a.dz, ld, a.n}, tp * BM,
          tq * BN, k0, k1);
    const int lane = threadIdx.x & 63;
    const int c0 = tp * BM + T::wave_p() + 4 * (lane >> 4), t0 = tq * BN + T::wave_q() + (lane & 15);
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int tok = t0 + 16 * j;
        if (tok >= a.n) continue;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int c = c0 + 16 * i;
            if (c >= a.d) continue;
            f32acc_t* o = reinterpret_cast<f32acc_t*>(out + (int64_t)tok * a.d + c);
            *o = first ? t.acc[i][j] : *o + t.acc[i][j];
        }
    }
}

__global__ __launch_bounds__(256) void ce_dh_join_kernel(const CeArgs a, int splits) {
    const int64_t total = (int64_t)a.n * a.d / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    f32acc_t s = reinterpret_cast<const f32acc_t*>(a.dh_part)[i];
    for (int k = 1; k < splits; ++k) s += reinterpret_cast<const f32acc_t*>(a.dh_part)[i + k * total];
    s *= *a.scale;
    if (a.grad_f32) reinterpret_cast<f32acc_t*>(a.dh)[i] = s;
    else reinterpret_cast<u32x2_t*>(a.dh)[i] = u32x2_t{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
}

// dw of a chunk = dz^T h.  P = h (width), Q = dz (vocabulary); tokens are the
// reduction index, which is dense in neither.
template <class T>
__global__ __launch_bounds__(T::THREADS) void ce_dw_kernel(const CeArgs a, int np, int nq, int vfirst, int count, int ld) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tp, tq;
    tile_of(np, nq, &tp, &tq);
    constexpr int BM = T::P_BYTES / 128, BN = T::Q_BYTES / 128;
    const int padded = (count + 63) / 64 * 64;
    const float scale = *a.scale;
    T t;
    t.run(lds, Operand{a.h, a.h_stride, a.d}, Operand{a.dz, ld, padded}, tp * BM, tq * BN, 0, a.n);
    const int lane = threadIdx.x & 63;
    const int c0 = tp * BM + T::wave_p() + 4 * (lane >> 4), v0 = tq * BN + T::wave_q() + (lane & 15);
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int v = v0 + 16 * j;
        if (v >= count) continue;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int c = c0 + 16 * i;
            if (c >= a.d) continue;
            const int64_t at = (int64_t)(vfirst + v) * a.d + c;
            const f32acc_t s = t.acc[i][j] * scale;
            if (a.grad_f32) *reinterpret_cast<f32acc_t*>(static_cast<float*>(a.dw) + at) = s;
            else *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.dw) + at) = u32x2_t{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
        }
    }
}

__global__ __launch_bounds__(256) void ce_zero_kernel(uint32_t* p, int64_t words) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < words) p[i] = 0u;
}

template <bool PT, bool QT>
using Large = TileProduct<256, 256, 2, 4, PT, QT>;
template <bool PT, bool QT>
using Small = TileProduct<128, 128, 2, 2, PT, QT>;
template <bool PT, bool QT>
using Few = TileProduct<64, 32, 4, 1, PT, QT>;

// The tile shape for `q` rows along Q and `p` along P.
enum Shape { LARGE, SMALL, FEW };
Shape shape_for(int64_t p, int64_t q) {
    if (q <= 32) return FEW;
    return ceil_div(p, 256) * ceil_div(q, 256) >= 192 ? LARGE : SMALL;
}
constexpr int kBM[3] = {256, 128, 64}, kBN[3] = {256, 128, 32}, kWM[3] = {2, 2, 4};

}  // namespace

int ce_parts(int n, int v) {
    const Shape s = shape_for(v, n);
    return (int)ceil_div(v, kBM[s]) * kWM[s];
}

CePlan ce_plan(int n, int d, int v) {
    CePlan p;
    n = std::max(n, 1);
    // dz of a chunk takes at most 256 MiB, the size of the memory-side cache
    const int64_t most = std::max<int64_t>(256, ((int64_t)128 << 20) / n / 256 * 256);
    const int64_t chunks = ceil_div(v, most);
    p.chunk = (int)(ceil_div(ceil_div(v, chunks), 256) * 256);
    const Shape s = shape_for(d, n);
    const int64_t tiles = ceil_div(d, kBM[s]) * ceil_div(n, kBN[s]);
    // enough workgroups for every CU, and at least 8 steps each
    const int64_t want = std::max<int64_t>(1, 512 / tiles);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(want, std::min(p.chunk, v) / (8 * GEMM_BK)));
    return p;
}

hipError_t launch_ce_fwd(const CeArgs& a, hipStream_t s) {
    const Shape sh = shape_for(a.v, a.n);
    const int np = (int)ceil_div(a.v, kBM[sh]), nq = (int)ceil_div(a.n, kBN[sh]);
    const dim3 g((unsigned)(np * nq));
    if (sh == LARGE) LRS_LAUNCH(K_LM_CE_STATS, (ce_stats_kernel<Large<false, false>>), g, dim3(512), 0, s, a, np, nq);
    else if (sh == SMALL) LRS_LAUNCH(K_LM_CE_STATS, (ce_stats_kernel<Small<false, false>>), g, dim3(256), 0, s, a, np, nq);
    else LRS_LAUNCH(K_LM_CE_STATS, (ce_stats_kernel<Few<false, false>>), g, dim3(256), 0, s, a, np, nq);
    LRS_LAUNCH(K_LM_CE_JOIN, ce_join_kernel, dim3((unsigned)ceil_div(a.n, 16)), dim3(1024), 0, s, a, ce_parts(a.n, a.v));
    return hipGetLastError();
}

hipError_t launch_ce_bwd(const CeArgs& a, hipStream_t s) {
    if (a.n == 0) {  // no token: dw is zero, and there is no dh
        const int64_t words = (int64_t)a.v * a.d * (a.grad_f32 ? 4 : 2) / 4;
        LRS_LAUNCH(K_CLEAR, ce_zero_kernel, dim3((unsigned)ceil_div(words, 256)), dim3(256), 0, s, (uint32_t*)a.dw, words);
        return hipGetLastError();
    }
    const CePlan pl = ce_plan(a.n, a.d, a.v);
    LRS_LAUNCH(K_LM_CE_JOIN, ce_scale_kernel, dim3(1), dim3(1024), 0, s, a);
    int used = 1;  // ranges of the first chunk, which is the longest
    for (int v0 = 0; v0 < a.v; v0 += pl.chunk) {
        const int count = std::min(pl.chunk, a.v - v0), ld = pl.chunk;
        {
            const Shape sh = shape_for(count, a.n);
            const int np = (int)ceil_div(count, kBM[sh]), nq = (int)ceil_div(a.n, kBN[sh]);
            const dim3 g((unsigned)(np * nq));
            if (sh == LARGE) LRS_LAUNCH(K_LM_CE_DZ, (ce_dz_kernel<Large<false, false>>), g, dim3(512), 0, s, a, np, nq, v0, count, ld);
            else if (sh == SMALL) LRS_LAUNCH(K_LM_CE_DZ, (ce_dz_kernel<Small<false, false>>), g, dim3(256), 0, s, a, np, nq, v0, count, ld);
            else LRS_LAUNCH(K_LM_CE_DZ, (ce_dz_kernel<Few<false, false>>), g, dim3(256), 0, s, a, np, nq, v0, count, ld);
        }
        {
            const Shape sh = shape_for(a.d, a.n);
            const int np = (int)ceil_div(a.d, kBM[sh]), nq = (int)ceil_div(a.n, kBN[sh]);
            const int range = (int)(ceil_div(ceil_div(count, pl.splits), GEMM_BK) * GEMM_BK), n_split = (int)ceil_div(count, range);
            if (v0 == 0) used = n_split;
            const dim3 g((unsigned)(np * nq * n_split));
            if (sh == LARGE) LRS_LAUNCH(K_LM_CE_DH, (ce_dh_kernel<Large<true, false>>), g, dim3(512), 0, s, a, np, nq, v0, count, ld, range, v0 == 0);
            else if (sh == SMALL) LRS_LAUNCH(K_LM_CE_DH, (ce_dh_kernel<Small<true, false>>), g, dim3(256), 0, s, a, np, nq, v0, count, ld, range, v0 == 0);
            else LRS_LAUNCH(K_LM_CE_DH, (ce_dh_kernel<Few<true, false>>), g, dim3(256), 0, s, a, np, nq, v0, count, ld, range, v0 == 0);
        }
        {
            const bool large = shape_for(a.d, std::max(count, 33)) == LARGE;
            const int b = large ? 256 : 128, np = (int)ceil_div(a.d, b), nq = (int)ceil_div(count, b);
            const dim3 g((unsigned)(np * nq));
            if (large) LRS_LAUNCH(K_LM_CE_DW, (ce_dw_kernel<Large<true, true>>), g, dim3(512), 0, s, a, np, nq, v0, count, ld);
            else LRS_LAUNCH(K_LM_CE_DW, (ce_dw_kernel<Small<true, true>>), g, dim3(256), 0, s, a, np, nq, v0, count, ld);
        }
    }
    LRS_LAUNCH(K_LM_CE_JOIN, ce_dh_join_kernel, dim3((unsigned)ceil_div((int64_t)a.n * a.d / 4, 256)), dim3(256), 0, s, a, used);
    return hipGetLastError();
}

}  // namespace lrs
