// lm_embed.hip -- the embedding lookup with its scale, and its gradient.
//
//   out_t = scale w[tok_t];   dw_v = scale sum_{t: tok_t = v} dout_t, in the order of the tokens.
//
// Both are bound by memory.  The gradient's sums go by tokens sorted by vocabulary row, so that each row is written once and
// no order depends on timing:
//   sort   every workgroup takes EMBED_ROWS rows of the vocabulary and looks at all tokens: it counts those of the rows before
//          its own (where its part of the order begins) and its own by row and wave, then places them.  Reading n tokens once for
//          each workgroup is little beside the n rows of dout: one launch does it all.
//   grad   a wave for each row writes it, zeros where it has no tokens; of rows with more than EMBED_RUN tokens, parts:
//          the sorted order is cut into runs of EMBED_RUN tokens, and a run sums what it holds of such a row.
//   join   adds the parts of such rows.
#include "lm.hpp"

namespace lrs {
namespace {

constexpr int WAVES = 16;  // of a sorting workgroup

// quads: groups of four columns; a thread has one of a token's.
template <class WT, class OT, bool TAIL>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const EmbedArgs a) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, quads = (a.d + 3) / 4, t = x / quads;
    if (t >= a.n) return;
    const int col = 4 * (int)(x % quads);
    const int64_t tok = a.tokens[t];
    float v[4];
    if (tok >= 0 && tok < a.v) {
        take<TAIL>(row_load<WT, TAIL>(static_cast<const WT*>(a.w) + tok * a.d, col, a.d), col, a.d, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= a.scale;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = tok < 0 ? 0.0f : __builtin_nanf("");
    }
    row_store<OT, TAIL>(static_cast<OT*>(a.out) + t * a.d, col, a.d, v);
}

__global__ __launch_bounds__(64 * WAVES) void embed_sort_kernel(const EmbedArgs a) {
    __shared__ int count[WAVES][EMBED_ROWS];  // a wave's tokens of each row, then where its next one of that row goes
    __shared__ int below[WAVES], sums[WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t lo = (int64_t)blockIdx.x * EMBED_ROWS, hi = min(lo + EMBED_ROWS, a.v);
    for (int i = threadIdx.x; i < WAVES * EMBED_ROWS; i += 64 * WAVES) (&count[0][0])[i] = 0;
    __syncthreads();
    // a wave's tokens are consecutive, so that the order within a row is theirs
    const int64_t per = (a.n + 64 * WAVES - 1) / (64 * WAVES) * 64, from = min(wave * per, a.n), to = min(from + per, a.n);
    int before = 0;
    for (int64_t i0 = from; i0 < to; i0 += 64 * 8) {
        int64_t t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = i0 + 64 * u + lane < to ? a.tokens[i0 + 64 * u + lane] : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (t[u] >= 0 && t[u] < lo) ++before;
            if (t[u] >= lo && t[u] < hi) atomicAdd(&count[wave][t[u] - lo], 1);
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) before += __shfl_xor(before, o);
    if (lane == 0) below[wave] = before;
    __syncthreads();
    // thread r: row r's place, from the rows before it and the workgroups before this one
    const int r = threadIdx.x;
    int mine = 0;
    if (r < EMBED_ROWS)
        for (int w = 0; w < WAVES; ++w) mine += count[w][r];
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int at = upto - mine;
    for (int w = 0; w < WAVES; ++w) at += below[w] + (w < wave ? sums[w] : 0);
    if (r < EMBED_ROWS) {
        if (lo + r < a.v) {
            a.start[lo + r] = at;
            if (lo + r == a.v - 1) a.start[a.v] = at + mine;
        }
        for (int w = 0; w < WAVES; ++w) {
            const int c = count[w][r];
            count[w][r] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t i0 = from; i0 < to; i0 += 64 * 8) {
        int64_t t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = i0 + 64 * u + lane < to ? a.tokens[i0 + 64 * u + lane] : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool here = t[u] >= lo && t[u] < hi;
            uint64_t same = __ballot(here);
            if (!same) continue;
            const int key = here ? (int)(t[u] - lo) : 0;
#pragma unroll
            for (int bit = 1; bit < EMBED_ROWS; bit <<= 1) {  // lanes with the same row
                const uint64_t m = __ballot((key & bit) != 0);
                same &= key & bit ? m : ~m;
            }
            const int rank = __popcll(same & ((1ull << lane) - 1));
            if (here) a.order[count[wave][key] + rank] = (int)(i0 + 64 * u + lane);
            wave_lds_sync();
            if (here && rank == 0) count[wave][key] += __popcll(same);
            wave_lds_sync();
        }
    }
}

// Adds rows order[p0..p1) of dout to s, eight of them on their way at a time.
template <class OT, bool TAIL>
__device__ __forceinline__ void add_rows(const EmbedArgs& a, int p0, int p1, int col, float* s) {
    for (int p = p0; p < p1; p += 8) {
        Quad<OT> q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t t = a.order[min(p + u, p1 - 1)];
            q[u] = row_load<OT, TAIL>(static_cast<const OT*>(a.dout) + t * a.dout_stride, col, a.d);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            float v[4];
            take<TAIL>(q[u], col, a.d, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += p + u < p1 ? v[i] : 0.0f;
        }
    }
}

// A row's gradient, rounded once; `add`: to what is there.
template <class GT, bool TAIL>
__device__ __forceinline__ void put_row(const EmbedArgs& a, int64_t row, int col, float* s) {
    GT* to = static_cast<GT*>(a.dw) + row * a.d;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.add) take<TAIL>(row_load<GT, TAIL>(to, col, a.d), col, a.d, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(a.scale, s[i], v[i]);
    row_store<GT, TAIL>(to, col, a.d, v);
}

// The first `runs` workgroups (of four) take the runs, the others the rows.
template <class OT, class GT, bool TAIL>
__global__ __launch_bounds__(256) void embed_grad_kernel(const EmbedArgs a, unsigned runs) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (blockIdx.x < runs) {
        const int64_t run = (int64_t)blockIdx.x * 4 + wave;
        const int total = a.start[a.v];
        if (run * EMBED_RUN >= total) return;
        const int p0 = (int)run * EMBED_RUN, p1 = min(p0 + EMBED_RUN, total);
        const int64_t head = a.tokens[a.order[p0]], tail = a.tokens[a.order[p1 - 1]];
        const int hs = a.start[head], he = a.start[head + 1], ts = a.start[tail], te = a.start[tail + 1];
        float* part = a.part + run * 2 * a.d;
        if (hs < p0 && he - hs > EMBED_RUN)
            for (int col = 4 * lane; col < a.d; col += 256) {
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                add_rows<OT, TAIL>(a, p0, min(he, p1), col, s);
                row_store<float, TAIL>(part, col, a.d, s);
            }
        if (ts >= p0 && te - ts > EMBED_RUN)
            for (int col = 4 * lane; col < a.d; col += 256) {
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                add_rows<OT, TAIL>(a, ts, p1, col, s);
                row_store<float, TAIL>(part + a.d, col, a.d, s);
            }
        return;
    }
    const int64_t row = (int64_t)(blockIdx.x - runs) * 4 + wave;
    if (row >= a.v) return;
    const int p0 = a.n > 0 ? a.start[row] : 0, p1 = a.n > 0 ? a.start[row + 1] : 0;
    if (p1 - p0 > EMBED_RUN || (a.add && p0 == p1)) return;
    for (int col = 4 * lane; col < a.d; col += 256) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        add_rows<OT, TAIL>(a, p0, p1, col, s);
        put_row<GT, TAIL>(a, row, col, s);
    }
}

// Rows of more than EMBED_RUN tokens: the workgroup of the run that such a row begins in adds its parts, wave w the w-th of each 16.
template <class GT, bool TAIL>
__global__ __launch_bounds__(64 * WAVES) void embed_join_kernel(const EmbedArgs a) {
    __shared__ float4 sum[WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t run = blockIdx.x;
    const int total = a.start[a.v];
    if (run * EMBED_RUN >= total) return;
    const int p0 = (int)run * EMBED_RUN, p1 = min(p0 + EMBED_RUN, total);
    const int64_t row = a.tokens[a.order[p1 - 1]];
    const int s0 = a.start[row], e0 = a.start[row + 1];
    if (s0 < p0 || e0 - s0 <= EMBED_RUN) return;
    const int parts = (e0 - 1) / EMBED_RUN - (int)run + 1;
    for (int c0 = 0; c0 < a.d; c0 += 256) {
        const int col = c0 + 4 * lane;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (col < a.d)
            for (int i = wave; i < parts; i += WAVES) {
                float v[4];
                const float* from = a.part + (run + i) * 2 * a.d + (i ? 0 : a.d);  // its first part is the end of a run
                take<TAIL>(row_load<float, TAIL>(from, col, a.d), col, a.d, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) s[k] += v[k];
            }
        sum[wave][lane] = make_float4(s[0], s[1], s[2], s[3]);
        __syncthreads();
        if (wave == 0 && col < a.d) {
            for (int w = 1; w < WAVES; ++w) {
                const float4 v = sum[w][lane];
                s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
            }
            put_row<GT, TAIL>(a, row, col, s);
        }
        __syncthreads();
    }
}

template <class WT, class OT>
void launch_fwd(const EmbedArgs& a, hipStream_t s) {
    const dim3 g((unsigned)ceil_div(a.n * ceil_div(a.d, 4), 256)), b(256);
    if (a.d % 4) LRS_LAUNCH(K_LM_EMBED, (embed_fwd_kernel<WT, OT, true>), g, b, 0, s, a);
    else LRS_LAUNCH(K_LM_EMBED, (embed_fwd_kernel<WT, OT, false>), g, b, 0, s, a);
}

template <class OT, class GT, bool TAIL>
void launch_grad(const EmbedArgs& a, hipStream_t s) {
    const int64_t runs = ceil_div(a.n, EMBED_RUN);
    const unsigned of_runs = (unsigned)ceil_div(runs, 4);
    if (a.n > 0) LRS_LAUNCH(K_LM_EMBED_SORT, embed_sort_kernel, dim3((unsigned)ceil_div(a.v, EMBED_ROWS)), dim3(64 * WAVES), 0, s, a);
    LRS_LAUNCH(K_LM_EMBED_GRAD, (embed_grad_kernel<OT, GT, TAIL>), dim3(of_runs + (unsigned)ceil_div(a.v, 4)), dim3(256), 0, s, a, of_runs);
    if (a.n > EMBED_RUN) LRS_LAUNCH(K_LM_EMBED_JOIN, (embed_join_kernel<GT, TAIL>), dim3((unsigned)runs), dim3(64 * WAVES), 0, s, a);
}
template <class OT, class GT>
void launch_grad_tail(const EmbedArgs& a, hipStream_t s) {
    if (a.d % 4) launch_grad<OT, GT, true>(a, s);
    else launch_grad<OT, GT, false>(a, s);
}

}  // namespace

hipError_t launch_embed_fwd(const EmbedArgs& a, bool w_f32, bool out_f32, hipStream_t s) {
    if (w_f32) {
        if (out_f32) launch_fwd<float, float>(a, s);
        else launch_fwd<float, uint16_t>(a, s);
    } else {
        if (out_f32) launch_fwd<uint16_t, float>(a, s);
        else launch_fwd<uint16_t, uint16_t>(a, s);
    }
    return hipGetLastError();
}

hipError_t launch_embed_bwd(const EmbedArgs& a, bool out_f32, bool grad_f32, hipStream_t s) {
    if (out_f32) {
        if (grad_f32) launch_grad_tail<float, float>(a, s);
        else launch_grad_tail<float, uint16_t>(a, s);
    } else {
        if (grad_f32) launch_grad_tail<uint16_t, float>(a, s);
        else launch_grad_tail<uint16_t, uint16_t>(a, s);
    }
    return hipGetLastError();
}

}  // namespace lrs
