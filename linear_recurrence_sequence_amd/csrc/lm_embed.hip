// lm_embed.hip -- the embedding lookup with its scale, and its gradient.
//
//   out_t = scale w[tok_t];   dw_v = scale sum_{t: tok_t = v} dout_t, in the order of the tokens.
//
// Both are bound by memory.  The gradient's sums go by tokens sorted by vocabulary row, so that each row is written once and
// no order depends on timing:
//   sort   every workgroup takes EMBED_ROWS rows of the vocabulary and looks at all tokens: it counts those of the rows before
//          its own (where its part of the order begins) and its own by row and wave, then places them, in one launch.  Every workgroup
//          reads all tokens twice, v / 32 bytes a token in all (4000 at v = 128000), mostly from the caches: as much as a row of dout of 2048 in
//          BF16, and more than one of 64.  32768 tokens with sort and join: v = 32000, 128000 and 256000 take 46, 59 and 70 us at d = 64 and
//          93, 169 and 273 at d = 2048, of which the writes of dw take most.
//   grad   a wave for each row writes it, zeros where it has no tokens; of rows with more than EMBED_RUN tokens, parts:
//          the sorted order is cut into runs of EMBED_RUN tokens, and a run sums what it holds of such a row.
//   join   adds the parts of such rows.
// 32768 tokens of a text's frequencies x 2048 in BF16, vocabulary 128000: lookup 56 us, sort 28, grad 138 (658 MB, 4.8 TB/s), join 7.
#include "lm.hpp"

namespace lrs {
namespace {

constexpr int BATCH = 4;   // groups of 256 columns (and tokens, in the gradient) whose loads of a wave are in flight together

// A wave takes BATCH * 256 columns of a token.
template <class WT, class OT, bool TAIL>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const EmbedArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.n) return;
    const int c0 = blockIdx.y * (256 * BATCH) + 4 * lane;
    const int64_t tok = a.tokens[t];
    const bool on = tok >= 0 && tok < a.v;
    const WT* row = static_cast<const WT*>(a.w) + (on ? tok : 0) * a.d;
    Quad<WT> q[BATCH];
#pragma unroll
    for (int c = 0; c < BATCH; ++c) q[c] = row_load<WT, TAIL>(row, min(c0 + 256 * c, a.d - 1), a.d);
#pragma unroll
    for (int c = 0; c < BATCH; ++c) {
        const int col = c0 + 256 * c;
        float v[4];
        take<TAIL>(q[c], col, a.d, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = on ? v[i] * a.scale : tok < 0 ? 0.0f : __builtin_nanf("");
        row_store<OT, TAIL>(static_cast<OT*>(a.out) + t * a.d, col, a.d, v);
    }
}

__global__ __launch_bounds__(64 * EMBED_WAVES) void embed_sort_kernel(const EmbedArgs a) {
    constexpr int WAVES = EMBED_WAVES;
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
            const uint64_t same = __ballot(here);
            if (!same) continue;
            const int key = here ? (int)(t[u] - lo) : 0;
            uint32_t s0 = (uint32_t)same, s1 = (uint32_t)(same >> 32);
#pragma unroll
            for (int bit = 0; 1 << bit < EMBED_ROWS; ++bit) {  // lanes with the same row: those whose bits all agree
                const uint64_t m = __ballot((key >> bit & 1) != 0);
                const uint32_t own = (uint32_t)-(key >> bit & 1);
                s0 &= ~((uint32_t)m ^ own), s1 &= ~((uint32_t)(m >> 32) ^ own);
            }
            const int rank = __builtin_amdgcn_mbcnt_hi(s1, __builtin_amdgcn_mbcnt_lo(s0, 0));
            if (here) a.order[count[wave][key] + rank] = (int)(i0 + 64 * u + lane);
            wave_lds_sync();
            if (here && rank == 0) count[wave][key] += __popc(s0) + __popc(s1);
            wave_lds_sync();
        }
    }
}

// Adds rows order[p0..p1) of dout, at most EMBED_RUN, to s: BATCH groups of 256 columns from c0 on.
template <class OT, bool TAIL>
__device__ __forceinline__ void add_rows(const EmbedArgs& a, int p0, int p1, int c0, float (&s)[BATCH][4]) {
    const int lane = threadIdx.x & 63, mine = a.order[min(p0 + lane, p1 - 1)];
#pragma unroll
    for (int c = 0; c < BATCH; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[c][i] = 0.0f;
    for (int p = 0; p < p1 - p0; p += BATCH) {
        Quad<OT> q[BATCH][BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int64_t t = __builtin_amdgcn_readlane(mine, min(p + u, p1 - p0 - 1));
            const OT* row = static_cast<const OT*>(a.dout) + t * a.dout_stride;
#pragma unroll
            for (int c = 0; c < BATCH; ++c) {
                const int col = c0 + 256 * c + 4 * lane;
                q[u][c] = row_load<OT, TAIL>(row, min(col, a.d - 1), a.d);
            }
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
#pragma unroll
            for (int c = 0; c < BATCH; ++c) {
                float v[4];
                take<TAIL>(q[u][c], c0 + 256 * c + 4 * lane, a.d, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[c][i] += p + u < p1 - p0 ? v[i] : 0.0f;
            }
    }
}

// A row's gradient, rounded once; `add`: to what is there.
template <class GT, bool TAIL>
__device__ __forceinline__ void put_row(const EmbedArgs& a, int64_t row, int col, const float* s) {
    GT* to = static_cast<GT*>(a.dw) + row * a.d;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.add) take<TAIL>(row_load<GT, TAIL>(to, col, a.d), col, a.d, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(a.scale, s[i], v[i]);
    row_store<GT, TAIL>(to, col, a.d, v);
}

// The first `runs` workgroups (of four) take the runs, the others rows: a wave every `waves`-th one, so that the frequent rows, which often stand
// side by side, are not one wave's.
template <class OT, class GT, bool TAIL>
__global__ __launch_bounds__(256) void embed_grad_kernel(const EmbedArgs a, unsigned runs, int waves) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float s[BATCH][4];
    if (blockIdx.x < runs) {
        const int64_t run = (int64_t)blockIdx.x * 4 + wave;
        const int total = a.start[a.v];
        if (run * EMBED_RUN >= total) return;
        const int p0 = (int)run * EMBED_RUN, p1 = min(p0 + EMBED_RUN, total);
        const int64_t head = a.tokens[a.order[p0]], tail = a.tokens[a.order[p1 - 1]];
        const int hs = a.start[head], he = a.start[head + 1], ts = a.start[tail], te = a.start[tail + 1];
        float* part = a.part + run * 2 * a.d;
        for (int c0 = 0; c0 < a.d; c0 += 256 * BATCH) {
            if (hs < p0 && he - hs > EMBED_RUN) {
                add_rows<OT, TAIL>(a, p0, min(he, p1), c0, s);
#pragma unroll
                for (int c = 0; c < BATCH; ++c) row_store<float, TAIL>(part, c0 + 256 * c + 4 * lane, a.d, s[c]);
            }
            if (ts >= p0 && te - ts > EMBED_RUN) {
                add_rows<OT, TAIL>(a, ts, p1, c0, s);
#pragma unroll
                for (int c = 0; c < BATCH; ++c) row_store<float, TAIL>(part + a.d, c0 + 256 * c + 4 * lane, a.d, s[c]);
            }
        }
        return;
    }
    const int first = (int)(blockIdx.x - runs) * 4 + wave;
    for (int64_t k0 = first; k0 < a.v; k0 += (int64_t)64 * waves) {
        // lane i: where the i-th of the next 64 rows begins and ends
        const int64_t r = min(k0 + (int64_t)lane * waves, a.v - 1);
        const int from = a.n > 0 ? a.start[r] : 0, to = a.n > 0 ? a.start[r + 1] : 0;
        for (int i = 0; i < 64 && k0 + (int64_t)i * waves < a.v; ++i) {
            const int64_t row = k0 + (int64_t)i * waves;
            const int p0 = __builtin_amdgcn_readlane(from, i), p1 = __builtin_amdgcn_readlane(to, i);
            if (p1 - p0 > EMBED_RUN || (a.add && p0 == p1)) continue;
            if (p0 == p1) {
                const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int col = 4 * lane; col < a.d; col += 256) row_store<GT, TAIL>(static_cast<GT*>(a.dw) + row * a.d, col, a.d, none);
                continue;
            }
            for (int c0 = 0; c0 < a.d; c0 += 256 * BATCH) {
                add_rows<OT, TAIL>(a, p0, p1, c0, s);
#pragma unroll
                for (int c = 0; c < BATCH; ++c)
                    if (c0 + 256 * c + 4 * lane < a.d) put_row<GT, TAIL>(a, row, c0 + 256 * c + 4 * lane, s[c]);
            }
        }
    }
}

// Rows of more than EMBED_RUN tokens: the workgroups of the run that such a row begins in add its parts, wave w the w-th of each JOIN_WAVES,
// 256 columns a workgroup.
constexpr int JOIN_WAVES = 4;
template <class GT, bool TAIL>
__global__ __launch_bounds__(64 * JOIN_WAVES) void embed_join_kernel(const EmbedArgs a) {
    __shared__ float4 sum[JOIN_WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.y * 256 + 4 * lane;
    const int64_t run = blockIdx.x;
    const int total = a.start[a.v];
    if (run * EMBED_RUN >= total) return;
    const int p0 = (int)run * EMBED_RUN, p1 = min(p0 + EMBED_RUN, total);
    const int64_t row = a.tokens[a.order[p1 - 1]];
    const int s0 = a.start[row], e0 = a.start[row + 1];
    if (s0 < p0 || e0 - s0 <= EMBED_RUN) return;
    const int parts = (e0 - 1) / EMBED_RUN - (int)run + 1;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i0 = wave; i0 < parts; i0 += 4 * JOIN_WAVES) {
        Quad<float> q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = min(i0 + u * JOIN_WAVES, parts - 1);
            q[u] = row_load<float, TAIL>(a.part + (run + i) * 2 * a.d + (i ? 0 : a.d), min(col, a.d - 1), a.d);  // its first part is the end of a run
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float v[4];
            take<TAIL>(q[u], col, a.d, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += i0 + u * JOIN_WAVES < parts ? v[k] : 0.0f;
        }
    }
    sum[wave][lane] = make_float4(s[0], s[1], s[2], s[3]);
    __syncthreads();
    if (wave > 0 || col >= a.d) return;
    for (int w = 1; w < JOIN_WAVES; ++w) {
        const float4 v = sum[w][lane];
        s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
    }
    put_row<GT, TAIL>(a, row, col, s);
}

template <class WT, class OT>
void launch_fwd(const EmbedArgs& a, hipStream_t s) {
    const dim3 g((unsigned)ceil_div(a.n, 4), (unsigned)ceil_div(a.d, 256 * BATCH)), b(256);
    if (a.d % 4) LRS_LAUNCH(K_LM_EMBED, (embed_fwd_kernel<WT, OT, true>), g, b, 0, s, a);
    else LRS_LAUNCH(K_LM_EMBED, (embed_fwd_kernel<WT, OT, false>), g, b, 0, s, a);
}

template <class OT, class GT, bool TAIL>
void launch_grad(const EmbedArgs& a, hipStream_t s) {
    const int64_t runs = ceil_div(a.n, EMBED_RUN);
    const unsigned of_runs = (unsigned)ceil_div(runs, 4);
    if (a.n > 0) LRS_LAUNCH(K_LM_EMBED_SORT, embed_sort_kernel, dim3((unsigned)ceil_div(a.v, EMBED_ROWS)), dim3(64 * EMBED_WAVES), 0, s, a);
    // 32768 tokens x 2048, vocabulary 128000: 2048, 4096, 8192, 16384 and all 32000 workgroups take 160, 149, 146, 140 and 139 us
    const unsigned of_rows = (unsigned)std::min<int64_t>(ceil_div(a.v, 4), 16384);
    LRS_LAUNCH(K_LM_EMBED_GRAD, (embed_grad_kernel<OT, GT, TAIL>), dim3(of_runs + of_rows), dim3(256), 0, s, a, of_runs, (int)of_rows * 4);
    if (a.n > EMBED_RUN) LRS_LAUNCH(K_LM_EMBED_JOIN, (embed_join_kernel<GT, TAIL>), dim3((unsigned)runs, (unsigned)ceil_div(a.d, 256)),
                                    dim3(64 * JOIN_WAVES), 0, s, a);
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
