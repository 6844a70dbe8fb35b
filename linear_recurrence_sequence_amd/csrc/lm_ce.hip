// lm_ce.hip -- softmax cross entropy of a linear head, forward and backward,
// without the logits in memory.
//
// For token t with hidden row h_t, vocabulary rows w_j and target y_t:
//   z_j = h_t . w_j, or c tanh(h_t . w_j / c) where logits are capped,
//   lse_t = log sum_j exp z_j,  loss_t = lse_t - z_{y_t} (0 where y_t < 0).
// The forward product's tiles end in a running maximum and sum of each token
// over the tile's vocabulary entries; a second small launch joins them.
// Backward, for the tokens that have a weight, vocabulary chunk by chunk: the
// logits are formed again, and
//   dz_j = (exp(z_j - lse_t) (dloss_t + dlse_t) - [j = y_t] dloss_t) (1 - tanh^2)
// is rounded to BF16 (the operand type of the matrix cores; a term is off by
// at most 2^-8 of it, independently of the others) into a buffer of one
// chunk, from which both products follow,
//   dh += dz w_chunk (FP32 sums kept over the chunks),  dw_chunk = dz^T h.
//
// Bound by the matrix cores for many tokens (2 n d v flops forward, 6 n d v
// backward): 8192 x 2048 x 128000 forward + backward 12.9 ms, 1.33 PFLOP/s, where
// four library products of the shape alone take 13.1; by reading w, and writing
// dw, for few: 16 x 1024 x 32000 forward 12.5 us, 5.2 TB/s, and a second launch.
#include "lm_ce_plan.hpp"
#include "lm_gemm.hpp"

namespace lrs {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// Which tile a workgroup takes.  Workgroups go to the 8 XCDs in turn, so each
// XCD is given a contiguous run of tiles, and a run walks over groups of 8
// tiles along q for each tile along p: what 32 neighbouring tiles read stays in
// the XCD's L2.
__device__ __forceinline__ void tile_of(int np, int nq, int b, int* p, int* q) {
    const int total = np * nq, xcd = b & 7, each = total >> 3, rest = total & 7;
    const int i = xcd * each + (xcd < rest ? xcd : rest) + (b >> 3);
    const int group = i / (8 * np), first = group * 8, size = nq - first < 8 ? nq - first : 8, in = i - first * np;
    *q = first + in % size;
    *p = in / size;
}

// tanh(z / cap) of four logits, in place, and its slope 1 - tanh^2.  Up to |x| = 1 the continued fraction
// x / (1 + x^2 / (3 + x^2 / (5 + ...))) to its sixth denominator, off by less than FP32's own
// rounding there; beyond, which a wave seldom meets, 1 - 2 q with q = 1 / (1 + e^2|x|), which near zero would
// keep the rounding of 1.  There the slope is 4 q (1 - q): formed from a tanh already rounded near 1 it would be off by
// 0.7% at |x| = 6.5 and zero from 9 on, where it is 6e-8.
__device__ __forceinline__ void cap_tanh(f32acc_t& z, f32acc_t& slope, float inv_cap) {
    float top = 0.0f;
    f32acc_t x, y;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        x[r] = z[r] * inv_cap;
        y[r] = x[r] * x[r];
        top = fmaxf(top, y[r]);
        z[r] = x[r] * fmaf(fmaf(21.0f, y[r], 1260.0f), y[r], 10395.0f) *
               __builtin_amdgcn_rcpf(fmaf(fmaf(y[r] + 210.0f, y[r], 4725.0f), y[r], 10395.0f));
        slope[r] = (1.0f - z[r]) * (1.0f + z[r]);
    }
    if (__ballot(top >= 1.0f)) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (!(y[r] < 1.0f)) {
                const float q = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(2.0f * LOG2E * fabsf(x[r])));
                z[r] = copysignf(1.0f - 2.0f * q, x[r]);
                slope[r] = 4.0f * q * (1.0f - q);
            }
    }
}

// Two (maximum, sum of 2^(z - maximum)) of base-2 logits as one.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x), base = fabsf(m) == __builtin_inff() ? 0.0f : m;
    return make_float2(m, a.y * __builtin_amdgcn_exp2f(a.x - base) + b.y * __builtin_amdgcn_exp2f(b.x - base));
}

// ------------------------------------------------------------- forward ---
// P = w (vocabulary), Q = h (tokens): a lane's results are 4 FM logits of each
// of FN tokens, so a token's maximum and sum are formed in registers, joined
// over the four lanes that share its column and then, through LDS, over the waves that
// share its tile.  w holds entries [vfirst, vfirst + a.v) here, whose tiles' statistics are
// parts from `part` on.
template <class T, bool CAP>
__global__ __launch_bounds__(T::THREADS) void ce_stats_kernel(const CeArgs a, int np, int nq, int vfirst, int part) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    __shared__ int target[T::TILE_Q];
    __shared__ float2 stat[T::WAVES_P][T::TILE_Q];
    constexpr int BM = T::TILE_P, BN = T::TILE_Q;
    int tp, tq;
    tile_of(np, nq, blockIdx.x, &tp, &tq);
    for (int i = threadIdx.x; i < BN; i += T::THREADS) {  // read after the barriers of the product
        const int64_t y = tq * BN + i < a.n ? a.target[tq * BN + i] - vfirst : -1;
        target[i] = y >= 0 && y < a.v ? (int)y : -1;
    }
    T t;
    t.run(lds, Operand{a.w, a.d, a.v}, Operand{a.h, a.h_stride, a.n}, tp * BM, tq * BN, 0, a.d);
    const int lane = threadIdx.x & 63, wave_p = (int)(threadIdx.x >> 6) / (T::WAVES / T::WAVES_P);
    const int v0 = tp * BM + 4 * (lane >> 4);
    if (CAP) {
        const float inv_cap = 1.0f / a.cap;
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                f32acc_t slope;
                cap_tanh(t.acc[i][j], slope, inv_cap);
                t.acc[i][j] *= a.cap;
            }
    }
    if ((tp + 1) * BM > a.v) {
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (v0 + T::row_p(i) + r >= a.v) t.acc[i][j][r] = -__builtin_inff();
    }
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int col = T::row_q(j) + (lane & 15), y = target[col] - v0;
        float top = -__builtin_inff();
        if (__ballot(y >= 0 && y < BM)) {  // seldom: a target among this tile's entries
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (y == T::row_p(i) + r) a.picked[tq * BN + col] = t.acc[i][j][r];
        }
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, t.acc[i][j][r]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = LOG2E * fmaxf(top, __shfl_xor(top, 32));
        // an infinite maximum is not subtracted: inf - inf would be NaN where the sum is inf or 0
        const float base = fabsf(top) == __builtin_inff() ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) sum += __builtin_amdgcn_exp2f(fmaf(t.acc[i][j][r], LOG2E, -base));
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (lane < 16) stat[wave_p][col] = make_float2(top, sum);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < BN; i += T::THREADS) {
        if (tq * BN + i >= a.n) continue;
        float2 s = stat[0][i];
#pragma unroll
        for (int k = 1; k < T::WAVES_P; ++k) s = join(s, stat[k][i]);
        reinterpret_cast<float2*>(a.part)[(int64_t)(part + tp) * a.n + tq * BN + i] = s;
    }
}

// Joins the tiles' maxima and sums of each token: 16 tokens a workgroup, 64
// lanes each, eight loads of a lane at a time.
__global__ __launch_bounds__(1024) void ce_join_kernel(const CeArgs a, int parts) {
    __shared__ float2 buf[16][17];
    const int c = threadIdx.x & 15, l = threadIdx.x >> 4, tok = blockIdx.x * 16 + c;
    float2 s = make_float2(-__builtin_inff(), 0.0f);
    if (tok < a.n)
        for (int i = l; i < parts; i += 64 * 8) {
            float2 o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] = i + 64 * k < parts ? reinterpret_cast<const float2*>(a.part)[(int64_t)(i + 64 * k) * a.n + tok]
                                          : make_float2(-__builtin_inff(), 0.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k) s = join(s, o[k]);
        }
    // four of a wave's lanes share a token, then the 16 waves do
    s = join(s, make_float2(__shfl_xor(s.x, 16), __shfl_xor(s.y, 16)));
    s = join(s, make_float2(__shfl_xor(s.x, 32), __shfl_xor(s.y, 32)));
    if ((l & 3) == 0) buf[l >> 2][c] = s;
    __syncthreads();
    if (l == 0)
#pragma unroll
        for (int i = 1; i < 16; ++i) s = join(s, buf[i][c]);
    if (l == 0 && tok < a.n) {
        const float base = fabsf(s.x) == __builtin_inff() ? 0.0f : s.x;
        const float more = __builtin_amdgcn_logf(s.y);
        const int64_t y = a.target[tok];
        a.lse[tok] = LN2 * (base + more);
        // The loss from differences in base 2, not from the rounded lse: it may be far smaller.
        // A target beyond the vocabulary has no loss: NaN says so.
        a.loss[tok] = y < 0 ? 0.0f : y < a.v ? LN2 * (fmaf(-a.picked[tok], LOG2E, base) + more) : __builtin_nanf("");
    }
}

// ------------------------------------------------------------ backward ---
// What the gradient takes from a token: dloss (0 where it does not count, NaN
// where its target does not exist) and the factor of its probabilities.
__device__ __forceinline__ void token_weights(const CeArgs& a, int tok, float* dl, float* c) {
    const int64_t y = a.target[tok];
    *dl = y < 0 ? 0.0f : y < a.v ? a.dloss[tok] : __builtin_nanf("");
    *c = a.dlse ? *dl + a.dlse[tok] : *dl;
}

// Row `from` of h to row `to` of the packed ones, by one wave.
__device__ __forceinline__ void pack_row(const CeArgs& a, int from, int to) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.h) + from * a.h_stride);
    u32x4_t* o = reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.packed) + (int64_t)to * a.d);
    for (int i = threadIdx.x & 63; i < a.d / 8; i += 64) o[i] = p[i];
}
// Tokens up to which the listing launch packs.  Backward of 1024 tokens x 1024 x 1000 43.0 us, 48.3 with a packing launch; of 512 38.1 and 40.7.
// Every workgroup walks all tokens for its list, so that the gain ends: of 2048 50.4 and 52.5, of 8192 126 and 128.
constexpr int LIST_PACKS = 1024;

// Lists the tokens that take part, those with a weight, in their order; the
// products run over these alone, so prompt and padding tokens cost nothing and
// whatever their rows hold stays out of dw.  Also the scale that dz is held at, the
// largest |dloss| or |dloss + dlse|: BF16 rounds dloss itself, and where all tokens
// weigh the same it would round each target's entry the same way, an error that no
// sum averages out; over the scale those entries are 1 - p.  Both products
// give it back.  One workgroup; up to 1024 tokens, a workgroup for 16 packed rows, each
// of which makes the list for itself and packs its rows (a launch less).
__global__ __launch_bounds__(1024) void ce_list_kernel(const CeArgs a) {
    __shared__ float best[16];
    __shared__ int count[16], source[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool writes = blockIdx.x == 0, packs = a.n <= LIST_PACKS;
    float top = 0.0f;
    for (int i = threadIdx.x; i < a.n; i += 1024) {
        float dl, c;
        token_weights(a, i, &dl, &c);
        const float w = fmaxf(fabsf(dl), fabsf(c));
        if (w < 0x1p100f) top = fmaxf(top, w);  // a weight that is not finite stays with its token
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) best[wave] = top;
    __syncthreads();
    for (int i = 0; i < 16; ++i) top = fmaxf(top, best[i]);
    const float scale = top < 0x1p-100f ? 1.0f : top, inv_scale = 1.0f / scale;
    int done = 0;
    for (int i0 = 0; i0 < a.n; i0 += 1024) {
        const int i = i0 + threadIdx.x;
        float dl = 0.0f, c = 0.0f;
        if (i < a.n) token_weights(a, i, &dl, &c);
        const bool in = dl != 0.0f || c != 0.0f;
        const uint64_t some = __ballot(in);
        __syncthreads();
        if (lane == 0) count[wave] = __popcll(some);
        __syncthreads();
        int before = done, all = 0;
        for (int k = 0; k < 16; ++k) {
            before += k < wave ? count[k] : 0;
            all += count[k];
        }
        done += all;
        if (i < a.n) {
            const int at = in ? before + __popcll(some & ((1ull << lane) - 1)) : -1;
            if (packs && in && at >> 4 == (int)blockIdx.x) source[at & 15] = i;
            if (!writes) continue;
            a.place[i] = at;
            if (in) {
                const int64_t y = a.target[i];
                a.list[at] = i;
                a.token[at] = CeToken{c * inv_scale, a.lse_in[i] * LOG2E, dl * inv_scale, y >= 0 && y < a.v ? (int)y : -1};
            }
        }
    }
    if (writes && threadIdx.x == 0) {
        *a.scale = scale;
        *a.active = done;
    }
    __syncthreads();
    const int row = (int)blockIdx.x * 16 + wave;
    if (packs && row < done) pack_row(a, source[wave], row);
}

// Rows of h that take part, packed: a wave a row.
__global__ __launch_bounds__(256) void ce_pack_kernel(const CeArgs a) {
    const int row = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row < *a.active) pack_row(a, a.list[row], row);
}

// dz / scale of vocabulary entries [vfirst, vfirst + count) for the listed tokens, BF16 [active, ld];
// columns from count to the next multiple of 64 are zeros.  With few tokens (a.few > 0)
// it is laid out [count, few], zeros beyond the listed tokens.
template <class T, bool CAP>
__global__ __launch_bounds__(T::THREADS) void ce_dz_kernel(const CeArgs a, int np, int vfirst, int count, int ld) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    __shared__ CeToken token[T::TILE_Q];
    constexpr int BM = T::TILE_P, BN = T::TILE_Q;
    const int m = *a.active, nq = ((a.few ? a.few : m) + BN - 1) / BN;
    if ((int)blockIdx.x >= np * nq) return;
    int tp, tq;
    tile_of(np, nq, blockIdx.x, &tp, &tq);
    for (int i = threadIdx.x; i < BN; i += T::THREADS)  // read after the barriers of the product
        if (tq * BN + i < m) token[i] = a.token[tq * BN + i];
    T t;
    t.run(lds, Operand{static_cast<const char*>(a.w) + (int64_t)vfirst * a.d * 2, a.d, count}, Operand{a.packed, a.d, m},
          tp * BM, tq * BN, 0, a.d);
    const int lane = threadIdx.x & 63, v0 = tp * BM + 4 * (lane >> 4), padded = (count + 63) / 64 * 64;
    const bool edge = (tp + 1) * BM > count;
    if (edge) {  // a probability of zero
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (v0 + T::row_p(i) + r >= count) t.acc[i][j][r] = -__builtin_inff();
    }
    const float inv_cap = CAP ? 1.0f / a.cap : 0.0f;
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int tok = tq * BN + T::row_q(j) + (lane & 15);
        if (tok >= (a.few ? a.few : m)) continue;
        const CeToken k = tok < m ? token[T::row_q(j) + (lane & 15)] : CeToken{0.0f, 0.0f, 0.0f, -1};
        const int y = k.target - vfirst - v0;  // no row of this wave where there is no target: rows + v0 + vfirst is not negative
        uint16_t* out = static_cast<uint16_t*>(a.dz) + (int64_t)tok * ld + v0;
        const bool hit = __ballot(y >= 0 && y < BM) != 0;  // seldom: a target among this tile's entries
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            float g[4];
            f32acc_t slope;
            if (CAP) cap_tanh(t.acc[i][j], slope, inv_cap);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                g[r] = __builtin_amdgcn_exp2f(fmaf(t.acc[i][j][r], CAP ? a.cap * LOG2E : LOG2E, -k.base)) * k.c;
            if (hit) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (y == T::row_p(i) + r) g[r] -= k.dl;
            }
            if (CAP) {
#pragma unroll
                for (int r = 0; r < 4; ++r) g[r] *= slope[r];
            }
            if (a.few) {
                if (tok >= m) g[0] = g[1] = g[2] = g[3] = 0.0f;
                uint16_t* t16 = static_cast<uint16_t*>(a.dz) + (int64_t)(v0 + T::row_p(i)) * a.few + tok;
                const uint32_t lo = pack_bf16x2(g[0], g[1]), hi = pack_bf16x2(g[2], g[3]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!edge || v0 + T::row_p(i) + r < count) t16[r * a.few] = (uint16_t)((r < 2 ? lo : hi) >> (16 * (r & 1)));
            } else if (!edge || v0 + T::row_p(i) < padded)
                *reinterpret_cast<u32x2_t*>(out + T::row_p(i)) = u32x2_t{pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3])};
        }
    }
}

// dh_part[s] (+)= dz w_chunk over range s of the chunk.  P = w (width; the
// reduction index is not the dense one), Q = dz (dense in it but with few tokens).
template <class T>
__global__ __launch_bounds__(T::THREADS) void ce_dh_kernel(const CeArgs a, int np, int vfirst, int count, int ld, int range,
                                                           int splits, int first) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    constexpr int BM = T::TILE_P, BN = T::TILE_Q;
    const int m = *a.active, nq = (m + BN - 1) / BN, tiles = np * nq;
    if ((int)blockIdx.x >= tiles * splits) return;
    int tp, tq;
    tile_of(np, nq, blockIdx.x % tiles, &tp, &tq);
    const int split = blockIdx.x / tiles, k0 = split * range, k1 = k0 + range < count ? k0 + range : count;
    float* out = a.dh_part + (int64_t)split * a.n * a.d;
    T t;
    t.run(lds, Operand{static_cast<const char*>(a.w) + (int64_t)vfirst * a.d * 2, a.d, a.d}, a.few ? Operand{a.dz, a.few, a.few} : Operand{a.dz, ld, m}, tp * BM,
          tq * BN, k0, k1);
    const int lane = threadIdx.x & 63;
    const int c0 = tp * BM + 4 * (lane >> 4), t0 = tq * BN + (lane & 15);
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int tok = t0 + T::row_q(j);
        if (tok >= m) continue;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int c = c0 + T::row_p(i);
            if (c >= a.d) continue;
            f32acc_t* o = reinterpret_cast<f32acc_t*>(out + (int64_t)tok * a.d + c);
            *o = first ? t.acc[i][j] : *o + t.acc[i][j];
        }
    }
}

// dh from the ranges' sums; zeros for the tokens that take no part.  Four
// columns a lane; of many ranges, G lanes sum every G-th each.
template <int G>
__global__ __launch_bounds__(256) void ce_dh_join_kernel(const CeArgs a, int splits) {
    constexpr int WIDE = 256 / G;
    __shared__ f32acc_t buf[G][WIDE];
    const int64_t part = (int64_t)a.n * a.d / 4, i = (int64_t)blockIdx.x * WIDE + threadIdx.x % WIDE;
    const int g = threadIdx.x / WIDE, line = a.d / 4;
    f32acc_t s = {0.f, 0.f, 0.f, 0.f};
    if (i < part) {
        const int at = a.place[i / line];
        if (at >= 0) {
            const f32acc_t* from = reinterpret_cast<const f32acc_t*>(a.dh_part) + (int64_t)at * line + i % line;
#pragma unroll 8
            for (int k = g; k < splits; k += G) s += from[k * part];
            s *= *a.scale;
        }
    }
    if (G > 1) {
        buf[g][threadIdx.x % WIDE] = s;
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int k = 1; k < G; ++k) s += buf[k][threadIdx.x];
    }
    if (i >= part) return;
    if (a.grad_f32) reinterpret_cast<f32acc_t*>(a.dh)[i] = s;
    else reinterpret_cast<u32x2_t*>(a.dh)[i] = u32x2_t{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
}

// dw of a chunk = dz^T h.  P = h (width), Q = dz (vocabulary); tokens are the
// reduction index, which is dense in neither.
template <class T>
__global__ __launch_bounds__(T::THREADS) void ce_dw_kernel(const CeArgs a, int np, int nq, int vfirst, int count, int ld) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    constexpr int BM = T::TILE_P, BN = T::TILE_Q;
    int tp, tq;
    tile_of(np, nq, blockIdx.x, &tp, &tq);
    const float scale = *a.scale;
    T t;
    t.run(lds, Operand{a.packed, a.d, a.d}, Operand{a.dz, ld, (count + 63) / 64 * 64}, tp * BM, tq * BN, 0, *a.active);
    const int lane = threadIdx.x & 63;
    const int c0 = tp * BM + 4 * (lane >> 4), v0 = tq * BN + (lane & 15);
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int v = v0 + T::row_q(j);
        if (v >= count) continue;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int c = c0 + T::row_p(i);
            if (c >= a.d) continue;
            const int64_t at = (int64_t)(vfirst + v) * a.d + c;
            const f32acc_t s = t.acc[i][j] * scale;
            if (a.grad_f32) *reinterpret_cast<f32acc_t*>(static_cast<float*>(a.dw) + at) = s;
            else *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.dw) + at) = u32x2_t{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
        }
    }
}

// dw of a chunk with few tokens (at most 32 KS): bound by writing dw.  A wave
// keeps the fragments of 64 columns of h in registers and walks over the
// vocabulary.  The workgroup's rows of dz, [count, 32 KS], are 8 KiB in a row: they are
// loaded as they lie, one piece ahead, and the fragments read from LDS (a fragment read
// from memory takes a line a lane: 70 us of the 108 us that 128 tokens x 2048 x 65536
// took).  The column
// of result r of fragment f in lane group g is chosen so that a lane's results of two
// fragments are 16 bytes of a row: 32 (f / 2) + 8 g + 4 (f % 2) + r.
template <int KS>
__global__ __launch_bounds__(256) void ce_dw_few_kernel(const CeArgs a, int vfirst, int count) {
    constexpr int U = 8 / KS, ROWS = U * 16, PIECES = KS * 4, PITCH = KS * 64 + 16;
    constexpr int LINE = 512 + 16;  // of 32 tokens' 256 columns of h, which stand in the same place first
    __shared__ __attribute__((aligned(16))) char lds[2 * ROWS * PITCH];
    static_assert(32 * LINE <= 2 * ROWS * PITCH, "32 tokens fit");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, m = *a.active;
    // an XCD writes whole rows: its workgroups take the columns of the same rows of dz
    const int cols = (a.d + 255) / 256, on = blockIdx.x >> 3, b0 = on % cols * 256, c0 = b0 + wave * 64;
    const int first = ((on / cols) * 8 + (blockIdx.x & 7)) * ROWS, stride = (int)gridDim.x / cols * ROWS;
    const float scale = *a.scale;
    bf16x8_t p[4][KS];
    u32x4_t slab[4];
    const auto fetch = [&](int ks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = i * 256 + threadIdx.x, tok = ks * 32 + at / 32, c = b0 + at % 32 * 8;
            slab[i] = tok < m && c < a.d ? *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.packed) + (int64_t)tok * a.d + c)
                                         : u32x4_t{0u, 0u, 0u, 0u};
        }
    };
    fetch(0);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = i * 256 + threadIdx.x;
            *reinterpret_cast<u32x4_t*>(lds + at / 32 * LINE + at % 32 * 16) = slab[i];
        }
        lds_barrier();
        if (ks + 1 < KS) fetch(ks + 1);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            // the transposing read: lane s of 16 reads 4 columns of one of 4 tokens and receives its own
            // column of all four; its own is the s % 4-th of the s / 4-th such four
            typedef __attribute__((address_space(3))) s16x4_t lds4;
            const int s = lane & 15, tok = 8 * g + (s >> 2), c = wave * 64 + 32 * (f / 2) + 8 * (s & 3) + 4 * (f % 2);
            const char* from = lds + tok * LINE + c * 2;
            s16x4_t v[2];
            v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)from);
            v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(from + 4 * LINE));
            p[f][ks] = __builtin_bit_cast(bf16x8_t, v);
        }
        lds_barrier();
    }
    const u32x4_t* dz = static_cast<const u32x4_t*>(a.dz);
    u32x4_t x[2];
    const auto load = [&](int row) {  // rows beyond the last are read as the last, and not stored
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = i * 256 + threadIdx.x, r = row + at / PIECES;
            x[i] = dz[(int64_t)(r < count ? r : count - 1) * PIECES + at % PIECES];
        }
    };
    const auto store = [&](const char* from, int row, bool whole) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = row + u * 16 + (lane & 15);
            f32acc_t c[4] = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const bf16x8_t q = *reinterpret_cast<const bf16x8_t*>(from + (u * 16 + (lane & 15)) * PITCH + (ks * 4 + g) * 16);
#pragma unroll
                for (int f = 0; f < 4; ++f) c[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[f][ks], q, c[f], 0, 0, 0);
            }
            if (!whole && v >= count) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = c0 + 32 * h + 8 * g;
                if (!whole && col >= a.d) continue;
                const f32acc_t y = c[2 * h] * scale, z = c[2 * h + 1] * scale;
                const int64_t at = (int64_t)(vfirst + v) * a.d + col;
                if (a.grad_f32) {
                    f32acc_t* o = reinterpret_cast<f32acc_t*>(static_cast<float*>(a.dw) + at);
                    o[0] = y;
                    o[1] = z;
                } else {
                    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.dw) + at) =
                        u32x4_t{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3])};
                }
            }
        }
    };
    load(first);
    int b = 0;
    for (int row = first; row < count; row += stride, b ^= 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = i * 256 + threadIdx.x;
            *reinterpret_cast<u32x4_t*>(lds + b * (ROWS * PITCH) + at / PIECES * PITCH + at % PIECES * 16) = x[i];
        }
        lds_barrier();
        load(row + stride);
        if (row + ROWS <= count && c0 + 64 <= a.d) store(lds + b * (ROWS * PITCH), row, true);
        else store(lds + b * (ROWS * PITCH), row, false);
    }
}

__global__ __launch_bounds__(256) void ce_zero_kernel(uint32_t* p, int64_t words) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) p[i] = 0u;
}

// Tiles.  256 x 256, one workgroup a CU: 8 waves where the tile ends in
// arithmetic on every result (two waves a SIMD share it), 4 where it ends in
// stores (their larger parts of the tile read a third less LDS).  128 x 128, two
// workgroups a CU, where the large ones would leave CUs idle.  64 x 32 for up to 32 tokens.
template <bool PT, bool QT>
using Wide = TileProduct<256, 256, 2, 4, PT, QT>;
template <bool PT, bool QT>
using Large = TileProduct<256, 256, 2, 2, PT, QT>;
template <bool PT, bool QT>
using Small = TileProduct<128, 128, 2, 2, PT, QT>;
template <bool PT, bool QT>
using Few = ThinProduct<64, 32, 4, 1, PT, QT>;
template <class T>
constexpr bool is_shape(Shape s) { return T::TILE_P == kBM[s] && T::TILE_Q == kBN[s]; }
static_assert(is_shape<Wide<false, false>>(LARGE) && is_shape<Large<true, true>>(LARGE) && is_shape<Small<true, true>>(SMALL) &&
              is_shape<Few<true, true>>(FEW) && CE_STEP == GEMM_BK, "the plan's tiles");
static_assert(Small<false, false>::THREADS == 256 && Few<false, false>::THREADS == 256, "threads of a tile that is not large");

}  // namespace

#define CE_SHAPES(shape, ID, GRID, KERNEL, BIG, PT, QT, ...)                                                                    \
    do {                                                                                                                       \
        if ((shape) == LARGE) LRS_LAUNCH(ID, (KERNEL(BIG<PT, QT>)), GRID, dim3(BIG<PT, QT>::THREADS), 0, s, __VA_ARGS__);         \
        else if ((shape) == SMALL) LRS_LAUNCH(ID, (KERNEL(Small<PT, QT>)), GRID, dim3(Small<PT, QT>::THREADS), 0, s, __VA_ARGS__); \
        else LRS_LAUNCH(ID, (KERNEL(Few<PT, QT>)), GRID, dim3(Few<PT, QT>::THREADS), 0, s, __VA_ARGS__);                          \
    } while (0)
#define CE_STATS(...) ce_stats_kernel<__VA_ARGS__, false>
#define CE_STATS_CAP(...) ce_stats_kernel<__VA_ARGS__, true>
#define CE_DZ(...) ce_dz_kernel<__VA_ARGS__, false>
#define CE_DZ_CAP(...) ce_dz_kernel<__VA_ARGS__, true>

hipError_t launch_ce_fwd(const CeArgs& a, hipStream_t s) {
    const int large = a.n <= 32 ? 0 : (int)large_rows(a.v, a.n, a.d);
    int part = 0;
    for (int v0 = 0; v0 < a.v;) {
        const int sh = a.n <= 32 ? FEW : v0 < large ? LARGE : SMALL;
        CeArgs p = a;
        p.w = static_cast<const char*>(a.w) + (int64_t)v0 * a.d * 2;
        // a launch over the threads that one may have is cut at a whole tile, so that the parts stay numbered by tiles
        p.v = (int)std::min<int64_t>((sh == LARGE ? large : a.v) - v0, ce_launch_rows((Shape)sh, sh == LARGE ? Wide<false, false>::THREADS : 256, a.n));
        const int np = (int)ceil_div(p.v, kBM[sh]), nq = (int)ceil_div(a.n, kBN[sh]);
        const dim3 g((unsigned)(np * nq));
        if (a.cap > 0.0f) CE_SHAPES(sh, K_LM_CE_STATS, g, CE_STATS_CAP, Wide, false, false, p, np, nq, v0, part);
        else CE_SHAPES(sh, K_LM_CE_STATS, g, CE_STATS, Wide, false, false, p, np, nq, v0, part);
        part += np;
        v0 += p.v;
    }
    LRS_LAUNCH(K_LM_CE_JOIN, ce_join_kernel, dim3((unsigned)ceil_div(a.n, 16)), dim3(1024), 0, s, a, part);
    return hipGetLastError();
}

// Grids are sized for all tokens; what lies beyond the listed ones exits at once.
hipError_t launch_ce_bwd(const CeArgs& args, hipStream_t s) {
    CeArgs a = args;
    if (a.n == 0) {  // no token: dw is zero, and there is no dh
        const int64_t words = (int64_t)a.v * a.d * (a.grad_f32 ? 4 : 2) / 4;
        LRS_LAUNCH(K_CLEAR, ce_zero_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(words, 256), 1 << 16)), dim3(256), 0, s, (uint32_t*)a.dw, words);
        return hipGetLastError();
    }
    const CePlan pl = ce_plan(a.n, a.d, a.v);
    a.few = pl.few;
    if (a.n <= LIST_PACKS) {
        LRS_LAUNCH(K_LM_CE_LIST, ce_list_kernel, dim3((unsigned)ceil_div(a.n, 16)), dim3(1024), 0, s, a);
    } else {
        LRS_LAUNCH(K_LM_CE_LIST, ce_list_kernel, dim3(1), dim3(1024), 0, s, a);
        LRS_LAUNCH(K_LM_CE_LIST, ce_pack_kernel, dim3((unsigned)ceil_div(a.n, 4)), dim3(256), 0, s, a);
    }
    for (int i = 0; i < ce_chunks(pl, a.v); ++i) {
        const CeChunk ch = ce_chunk(pl, a.v, i);
        const int v0 = ch.first, count = ch.count, splits = ch.splits, range = pl.range, ld = pl.chunk;
        const auto part_of = [&](int at) {  // the arguments with dz from entry `at` of the chunk on
            CeArgs p = a;
            p.dz = static_cast<uint16_t*>(a.dz) + (int64_t)at * (a.few ? a.few : 1);
            return p;
        };
        for (int at = 0, large = a.n <= 32 ? 0 : (int)large_rows(count, a.n, a.d); at < count;) {
            const int sh = a.n <= 32 ? FEW : at < large ? LARGE : SMALL, some = (sh == LARGE ? large : count) - at;
            const CeArgs p = part_of(at);
            const int np = (int)ceil_div(some, kBM[sh]);
            const dim3 g((unsigned)(np * ceil_div(pl.few ? pl.few : a.n, kBN[sh])));
            if (a.cap > 0.0f) CE_SHAPES(sh, K_LM_CE_DZ, g, CE_DZ_CAP, Wide, false, false, p, np, v0 + at, some, ld);
            else CE_SHAPES(sh, K_LM_CE_DZ, g, CE_DZ, Wide, false, false, p, np, v0 + at, some, ld);
            at += some;
        }
        {
            const int np = (int)ceil_div(a.d, kBM[pl.dh]);
            const dim3 g((unsigned)(np * ceil_div(a.n, kBN[pl.dh]) * splits));
            if (pl.dh == LARGE) LRS_LAUNCH(K_LM_CE_DH, (ce_dh_kernel<Large<true, false>>), g, dim3(Large<true, false>::THREADS), 0, s, a, np, v0, count, ld, range, splits, v0 == 0);
            else if (!pl.few) LRS_LAUNCH(K_LM_CE_DH, (ce_dh_kernel<Small<true, false>>), g, dim3(Small<true, false>::THREADS), 0, s, a, np, v0, count, ld, range, splits, v0 == 0);
            else if (pl.dh == SMALL) LRS_LAUNCH(K_LM_CE_DH, (ce_dh_kernel<Small<true, true>>), g, dim3(Small<true, true>::THREADS), 0, s, a, np, v0, count, ld, range, splits, v0 == 0);
            else LRS_LAUNCH(K_LM_CE_DH, (ce_dh_kernel<Few<true, true>>), g, dim3(Few<true, true>::THREADS), 0, s, a, np, v0, count, ld, range, splits, v0 == 0);
        }
        if (pl.few) {
            const int cols = (int)ceil_div(a.d, 256), rows = 4096 / pl.few;  // rows of dz a workgroup takes at a time
            const dim3 g((unsigned)(cols * 8 * std::max<int64_t>(1, std::min<int64_t>(ceil_div(count, 8 * rows), 64 / cols))));
            if (pl.few == 32) LRS_LAUNCH(K_LM_CE_DW, ce_dw_few_kernel<1>, g, dim3(256), 0, s, a, v0, count);
            else if (pl.few == 64) LRS_LAUNCH(K_LM_CE_DW, ce_dw_few_kernel<2>, g, dim3(256), 0, s, a, v0, count);
            else if (pl.few == 128) LRS_LAUNCH(K_LM_CE_DW, ce_dw_few_kernel<4>, g, dim3(256), 0, s, a, v0, count);
            else LRS_LAUNCH(K_LM_CE_DW, ce_dw_few_kernel<8>, g, dim3(256), 0, s, a, v0, count);
        } else {
            for (int at = 0, large = (int)large_rows(count, a.d, a.n); at < count;) {
                const int sh = at < large ? LARGE : SMALL, some = (sh == LARGE ? large : count) - at;
                const CeArgs p = part_of(at);
                const int np = (int)ceil_div(a.d, kBM[sh]), nq = (int)ceil_div(some, kBN[sh]);
                const dim3 g((unsigned)(np * nq));
                if (sh == LARGE) LRS_LAUNCH(K_LM_CE_DW, (ce_dw_kernel<Large<true, true>>), g, dim3(Large<true, true>::THREADS), 0, s, p, np, nq, v0 + at, some, ld);
                else LRS_LAUNCH(K_LM_CE_DW, (ce_dw_kernel<Small<true, true>>), g, dim3(Small<true, true>::THREADS), 0, s, p, np, nq, v0 + at, some, ld);
                at += some;
            }
        }
    }
    const int64_t quads = (int64_t)a.n * a.d / 4;
    // Eight lanes a sum against one: of 125 ranges (16 x 512 x 32000) the backward takes 36.3 us against 39.8, of 63 (16 x 1024 x 32000)
    // 49.4 against 51.5; of 12 (600 x 1024 x 32000) 173.9 against 171.1, of 8 (2048 x 1024 x 32000) 389 against 384; between them either way, by 1%.
    if (pl.splits >= 16) LRS_LAUNCH(K_LM_CE_JOIN, ce_dh_join_kernel<8>, dim3((unsigned)ceil_div(quads, 32)), dim3(256), 0, s, a, pl.splits);
    else LRS_LAUNCH(K_LM_CE_JOIN, ce_dh_join_kernel<1>, dim3((unsigned)ceil_div(quads, 256)), dim3(256), 0, s, a, pl.splits);
    return hipGetLastError();
}

}  // namespace lrs
