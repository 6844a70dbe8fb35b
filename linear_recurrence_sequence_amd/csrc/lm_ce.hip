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
__device__ __forceinline__ void tile_of(int np, int nq, int b, int* p, int* q) {
    const int total = np * nq, xcd = b & 7, each = total >> 3, rest = total & 7;
    const int i = xcd * each + (xcd < rest ? xcd : rest) + (b >> 3);
    const int group = i / (8 * np), first = group * 8, size = nq - first < 8 ? nq - first : 8, in = i - first * np;
    *q = first + in % size;
    *p = in / size;
}

__device__ __forceinline__ float cap_tanh(float z, float inv_cap) {  // tanh(z / cap)
    return 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(2.0f * LOG2E * inv_cap * z));
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
// share its tile.
template <class T, bool CAP>
__global__ __launch_bounds__(T::THREADS) void ce_stats_kernel(const CeArgs a, int np, int nq) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    __shared__ int target[T::TILE_Q];
    __shared__ float2 stat[T::WAVES_P][T::TILE_Q];
    constexpr int BM = T::TILE_P, BN = T::TILE_Q;
    int tp, tq;
    tile_of(np, nq, blockIdx.x, &tp, &tq);
    for (int i = threadIdx.x; i < BN; i += T::THREADS) {  // read after the barriers of the product
        const int64_t y = tq * BN + i < a.n ? a.target[tq * BN + i] : -1;
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
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) t.acc[i][j][r] = a.cap * cap_tanh(t.acc[i][j][r], inv_cap);
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
        float top = -__builtin_inff(), hit = 0.0f;
        bool mine = false;
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float z = t.acc[i][j][r];
                if (y == T::row_p(i) + r) hit = z, mine = true;
                top = fmaxf(top, z);
            }
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
        if (mine) a.picked[tq * BN + col] = hit;
        if (lane < 16) stat[wave_p][col] = make_float2(top, sum);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < BN; i += T::THREADS) {
        if (tq * BN + i >= a.n) continue;
        float2 s = stat[0][i];
#pragma unroll
        for (int k = 1; k < T::WAVES_P; ++k) s = join(s, stat[k][i]);
        reinterpret_cast<float2*>(a.part)[(int64_t)tp * a.n + tq * BN + i] = s;
    }
}

// Joins the tiles' maxima and sums of each token: 16 tokens a workgroup, 64
// lanes each, eight loads of a lane at a time.
__global__ __launch_bounds__(1024) void ce_join_kernel(const CeArgs a, int parts) {
    __shared__ float2 buf[64][17];
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
    buf[l][c] = s;
    __syncthreads();
    for (int o = 32; o > 0; o >>= 1) {
        if (l < o) buf[l][c] = s = join(s, buf[l + o][c]);
        __syncthreads();
    }
    if (l == 0 && tok < a.n) {
        const float base = fabsf(s.x) == __builtin_inff() ? 0.0f : s.x;
        const float lse = LN2 * (base + __builtin_amdgcn_logf(s.y));
        const int64_t y = a.target[tok];
        a.lse[tok] = lse;
        // a target beyond the vocabulary has no loss: NaN says so
        a.loss[tok] = y < 0 ? 0.0f : y < a.v ? lse - a.picked[tok] : __builtin_nanf("");
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

// Lists the tokens that take part, those with a weight, in their order; the
// products run over these alone, so prompt and padding tokens cost nothing and
// whatever their rows hold stays out of dw.  Also the scale that dz is held at, the
// largest |dloss| or |dloss + dlse|: BF16 rounds dloss itself, and where all tokens
// weigh the same it would round each target's entry the same way, an error that no
// sum averages out; over the scale those entries are 1 - p.  Both products
// give it back.  One workgroup.
__global__ __launch_bounds__(1024) void ce_list_kernel(const CeArgs a) {
    __shared__ float best[16];
    __shared__ int count[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
            a.place[i] = at;
            if (in) {
                const int64_t y = a.target[i];
                a.list[at] = i;
                a.token[at] = CeToken{c * inv_scale, a.lse_in[i] * LOG2E, dl * inv_scale, y >= 0 && y < a.v ? (int)y : -1};
            }
        }
    }
    if (threadIdx.x == 0) {
        *a.scale = scale;
        *a.active = done;
    }
}

// Rows of h that take part, packed: a wave a row, 8 elements a lane at a time.
__global__ __launch_bounds__(256) void ce_pack_kernel(const CeArgs a) {
    const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (row >= *a.active) return;
    const u32x4_t* from = reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.h) + a.list[row] * a.h_stride);
    u32x4_t* to = reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.packed) + (int64_t)row * a.d);
    for (int i = lane; i < a.d / 8; i += 64) to[i] = from[i];
}

// dz / scale of vocabulary entries [vfirst, vfirst + count) for the listed tokens, BF16 [active, ld];
// columns from count to the next multiple of 64 are zeros.
template <class T, bool CAP>
__global__ __launch_bounds__(T::THREADS) void ce_dz_kernel(const CeArgs a, int np, int vfirst, int count, int ld) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    __shared__ CeToken token[T::TILE_Q];
    constexpr int BM = T::TILE_P, BN = T::TILE_Q;
    const int m = *a.active, nq = (m + BN - 1) / BN;
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
        if (tok >= m) continue;
        const CeToken k = token[T::row_q(j) + (lane & 15)];
        const int y = k.target - vfirst - v0;  // no row of this wave where there is no target: rows + v0 + vfirst is not negative
        uint16_t* out = static_cast<uint16_t*>(a.dz) + (int64_t)tok * ld + v0;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            float g[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float z = t.acc[i][j][r], slope = 1.0f;
                if (CAP) {
                    const float th = cap_tanh(z, inv_cap);
                    z = a.cap * th;
                    slope = (1.0f - th) * (1.0f + th);
                }
                g[r] = __builtin_amdgcn_exp2f(fmaf(z, LOG2E, -k.base)) * k.c;
                if (y == T::row_p(i) + r) g[r] -= k.dl;
                if (CAP) g[r] *= slope;
            }
            if (!edge || v0 + T::row_p(i) < padded)
                *reinterpret_cast<u32x2_t*>(out + T::row_p(i)) = u32x2_t{pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3])};
        }
    }
}

// dh_part[s] (+)= dz w_chunk over range s of the chunk.  P = w (width; the
// reduction index is not the dense one), Q = dz.
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
    t.run(lds, Operand{static_cast<const char*>(a.w) + (int64_t)vfirst * a.d * 2, a.d, a.d}, Operand{a.dz, ld, m}, tp * BM,
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

// dh from the ranges' sums; zeros for the tokens that take no part.  A wave a row.
__global__ __launch_bounds__(256) void ce_dh_join_kernel(const CeArgs a, int splits) {
    const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (row >= a.n) return;
    const int at = a.place[row];
    const float scale = *a.scale;
    const int64_t part = (int64_t)a.n * a.d / 4;
    const f32acc_t* from = reinterpret_cast<const f32acc_t*>(a.dh_part) + (int64_t)at * (a.d / 4);
    for (int i = lane; i < a.d / 4; i += 64) {
        f32acc_t s = {0.f, 0.f, 0.f, 0.f};
        if (at >= 0) {
            s = from[i];
#pragma unroll 8
            for (int k = 1; k < splits; ++k) s += from[i + k * part];
            s *= scale;
        }
        const int64_t o = (int64_t)row * (a.d / 4) + i;
        if (a.grad_f32) reinterpret_cast<f32acc_t*>(a.dh)[o] = s;
        else reinterpret_cast<u32x2_t*>(a.dh)[o] = u32x2_t{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    }
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

__global__ __launch_bounds__(256) void ce_zero_kernel(uint32_t* p, int64_t words) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < words) p[i] = 0u;
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

enum Shape { LARGE, SMALL, FEW };
constexpr int kBM[3] = {256, 128, 64}, kBN[3] = {256, 128, 32};

constexpr int64_t kMostDz = (int64_t)128 << 20;  // elements of dz held at once

// Time of a product of p x q results over k, in microseconds: rounds of
// workgroups times steps of 64, with three steps' worth of start and end a tile.
// A round's step takes 1.54 us with large tiles and 1.04 us with small ones (half the
// flops), both measured over long k with every CU busy.
double product_us(Shape s, int64_t p, int64_t q, int64_t k) {
    const int64_t tiles = ceil_div(p, kBM[s]) * ceil_div(q, kBN[s]), slots = s == LARGE ? 256 : 512;
    return (double)ceil_div(tiles, slots) * (double)(ceil_div(k, GEMM_BK) + 3) * (s == LARGE ? 1.54 : 1.04);
}
Shape shape_for(int64_t p, int64_t q, int64_t k) {
    return product_us(LARGE, p, q, k) <= product_us(SMALL, p, q, k) ? LARGE : SMALL;
}

}  // namespace

// Tile of the forward product.
static Shape stats_shape(int n, int d, int v) { return n <= 32 ? FEW : shape_for(v, n, d); }

int ce_parts(int n, int d, int v) { return (int)ceil_div(v, kBM[stats_shape(n, d, v)]); }

// Chunks of the vocabulary, tiles and the ranges that dh is summed over: the
// cheapest by product_us and the bytes of dh's partial sums, over the chunk
// counts from the least that the buffer of dz allows.
CePlan ce_plan(int n, int d, int v) {
    n = std::max(n, 1);
    const int64_t most = std::max<int64_t>(256, kMostDz / n / 256 * 256), least = ceil_div(v, most);
    CePlan best{};
    double best_us = 0.0;
    for (int64_t chunks = least; chunks < least + 8; ++chunks) {
        const int64_t chunk = ceil_div(ceil_div(v, chunks), 256) * 256, count = std::min<int64_t>(chunk, v);
        CePlan p{};
        p.chunk = (int)chunk;
        p.dz = n <= 32 ? FEW : shape_for(count, n, d);
        p.dw = shape_for(d, count, n);
        double us = n <= 32 ? 0.0 : product_us((Shape)p.dz, count, n, d);
        us += product_us((Shape)p.dw, d, count, n);
        double dh_us = 0.0;
        for (int s = LARGE; s <= FEW; ++s) {
            if ((s == FEW) != (n <= 32)) continue;
            for (int splits = 1; splits <= 16 && (splits == 1 || count / splits >= 8 * GEMM_BK); ++splits) {
                // the partial sums are written, and read by the next chunk or the last launch
                const double t = product_us((Shape)s, d, (int64_t)n * splits, ceil_div(count, splits)) + (double)splits * n * d * 8 / 4.5e6;
                if (dh_us == 0.0 || t < dh_us) dh_us = t, p.dh = s, p.splits = splits;
            }
        }
        us = (us + dh_us) * (double)ceil_div(v, chunk);
        if (best_us == 0.0 || us < best_us) best_us = us, best = p;
    }
    return best;
}

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
#define CE_DH(...) ce_dh_kernel<__VA_ARGS__>

hipError_t launch_ce_fwd(const CeArgs& a, hipStream_t s) {
    const Shape sh = stats_shape(a.n, a.d, a.v);
    const int np = (int)ceil_div(a.v, kBM[sh]), nq = (int)ceil_div(a.n, kBN[sh]);
    const dim3 g((unsigned)(np * nq));
    if (a.cap > 0.0f) CE_SHAPES(sh, K_LM_CE_STATS, g, CE_STATS_CAP, Wide, false, false, a, np, nq);
    else CE_SHAPES(sh, K_LM_CE_STATS, g, CE_STATS, Wide, false, false, a, np, nq);
    LRS_LAUNCH(K_LM_CE_JOIN, ce_join_kernel, dim3((unsigned)ceil_div(a.n, 16)), dim3(1024), 0, s, a, np);
    return hipGetLastError();
}

// Grids are sized for all tokens; what lies beyond the listed ones exits at once.
hipError_t launch_ce_bwd(const CeArgs& a, hipStream_t s) {
    if (a.n == 0) {  // no token: dw is zero, and there is no dh
        const int64_t words = (int64_t)a.v * a.d * (a.grad_f32 ? 4 : 2) / 4;
        LRS_LAUNCH(K_CLEAR, ce_zero_kernel, dim3((unsigned)ceil_div(words, 256)), dim3(256), 0, s, (uint32_t*)a.dw, words);
        return hipGetLastError();
    }
    const CePlan pl = ce_plan(a.n, a.d, a.v);
    const dim3 rows((unsigned)ceil_div(a.n, 4));
    LRS_LAUNCH(K_LM_CE_LIST, ce_list_kernel, dim3(1), dim3(1024), 0, s, a);
    LRS_LAUNCH(K_LM_CE_LIST, ce_pack_kernel, rows, dim3(256), 0, s, a);
    int used = 1;  // ranges of the first chunk, which is the longest
    for (int v0 = 0; v0 < a.v; v0 += pl.chunk) {
        const int count = std::min(pl.chunk, a.v - v0), ld = pl.chunk;
        {
            const int np = (int)ceil_div(count, kBM[pl.dz]);
            const dim3 g((unsigned)(np * ceil_div(a.n, kBN[pl.dz])));
            if (a.cap > 0.0f) CE_SHAPES(pl.dz, K_LM_CE_DZ, g, CE_DZ_CAP, Wide, false, false, a, np, v0, count, ld);
            else CE_SHAPES(pl.dz, K_LM_CE_DZ, g, CE_DZ, Wide, false, false, a, np, v0, count, ld);
        }
        {
            const int np = (int)ceil_div(a.d, kBM[pl.dh]);
            const int range = (int)(ceil_div(ceil_div(count, pl.splits), GEMM_BK) * GEMM_BK), splits = (int)ceil_div(count, range);
            if (v0 == 0) used = splits;
            const dim3 g((unsigned)(np * ceil_div(a.n, kBN[pl.dh]) * splits));
            CE_SHAPES(pl.dh, K_LM_CE_DH, g, CE_DH, Large, true, false, a, np, v0, count, ld, range, splits, v0 == 0);
        }
        {
            const int np = (int)ceil_div(a.d, kBM[pl.dw]), nq = (int)ceil_div(count, kBN[pl.dw]);
            const dim3 g((unsigned)(np * nq));
            if (pl.dw == LARGE) LRS_LAUNCH(K_LM_CE_DW, (ce_dw_kernel<Large<true, true>>), g, dim3(Large<true, true>::THREADS), 0, s, a, np, nq, v0, count, ld);
            else LRS_LAUNCH(K_LM_CE_DW, (ce_dw_kernel<Small<true, true>>), g, dim3(Small<true, true>::THREADS), 0, s, a, np, nq, v0, count, ld);
        }
    }
    LRS_LAUNCH(K_LM_CE_JOIN, ce_dh_join_kernel, rows, dim3(256), 0, s, a, used);
    return hipGetLastError();
}

}  // namespace lrs
