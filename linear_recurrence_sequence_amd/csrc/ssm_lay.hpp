// ssm_lay.hpp -- where a wave of the selective scan stands, and how it reads a
// chunk.
#pragma once

#include <type_traits>

#include "ssm.hpp"

namespace lrs {

template <int NG>
struct Lay {
    static constexpr int J = 64 / NG, CH = 2 * J, N4 = SSM_STATES * NG, Q = SSM_TOK / NG;
};

// The lane's number, formed anew: what is derived from it inside a loop stays there, where keeping a register for each of many addresses
// would cost more than a few integer operations a chunk.
__device__ __forceinline__ uint32_t fresh_lane() {
    uint32_t lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    __builtin_assume(lane < 64);
    return lane;
}

// f(std::bool_constant) for a condition that all lanes share: the two cases are compiled apart.
template <class F>
__device__ __forceinline__ void both_ways(bool uniform, F f) {
    if (uniform) f(std::true_type{});
    else f(std::false_type{});
}

// A wave's row and segment, its lane's part of the channels and states.
struct Place {
    int b, seg, gr, tile, c0;    // row, segment, group of b and c, tile of its channels, the lane's first channel
    int i;                       // first of the two channels that the lane loads: its own, or existing ones of its group
    bool ok0, ok1, odd;          // which of its channels exist; odd: the first is the second one loaded (a group's last, without a partner)
    int g, j;                    // the lane's group of states and pair of channels
};
template <int NG>
__device__ __forceinline__ Place place_of(const SsmArgs& a, int tile, int gr, int seg, int b) {
    const int lane = threadIdx.x & 63, end = (gr + 1) * a.per;
    Place p;
    p.b = b, p.seg = seg, p.gr = gr, p.tile = tile;
    p.g = lane / Lay<NG>::J, p.j = lane % Lay<NG>::J;
    p.c0 = gr * a.per + tile * Lay<NG>::CH + 2 * p.j;
    p.ok0 = p.c0 < end, p.ok1 = p.c0 + 1 < end;
    // Lanes without channels load their group's last ones: what those of another group hold, NaN say, must not reach this one's db and dc.
    p.i = max(min(p.c0, end - 2), gr * a.per);
    p.odd = p.c0 == p.i + 1 || a.per == 1;  // a group's only channel is loaded as the second
    return p;
}

// A loaded pair as the lane's own channels.
__device__ __forceinline__ float2 own(float2 v, const Place& p) { return make_float2(p.odd ? v.y : v.x, v.y); }

__device__ __forceinline__ int length_of(const SsmArgs& a, int b) {
    return a.lengths ? min(max(a.lengths[b], 0), a.length) : a.length;
}

// Bit t: token t0 + t of row b starts a sequence, in the padding too.
__device__ __forceinline__ uint32_t resets_of(const SsmArgs& a, int b, int t0) {
    if (!a.reset) return 0u;
    const int t = t0 + (threadIdx.x & 63);
    const bool r = t < min(t0 + SSM_TOK, a.length) && a.reset[(int64_t)b * a.length + t] != 0;
    return (uint32_t)__ballot(r);
}

// A chunk's rows of one tensor: a uniform base, and a lane's offset in bytes from a row number below 16 and a
// distance below 2^22 elements (SSM_MOST_STRIDE).
template <class T>
__device__ __forceinline__ const char* rows_at(const void* p, int64_t row, int64_t stride) {
    return static_cast<const char*>(p) + row * stride * sizeof(T);
}
template <class T>
__device__ __forceinline__ char* rows_at(void* p, int64_t row, int64_t stride) {
    return static_cast<char*>(p) + row * stride * sizeof(T);
}
template <class T>
__device__ __forceinline__ uint32_t row_off(int r, int64_t stride, int col) {
    return (__umul24((uint32_t)r, (uint32_t)stride) + (uint32_t)col) * sizeof(T);
}
// Of a record of states [n][d].
__device__ __forceinline__ uint32_t state_off(const SsmArgs& a, int n, int col) { return ((uint32_t)(n * a.d) + (uint32_t)col) * 4; }

// What b or c hold for a chunk, a lane's part: element e * 64 + lane of [SSM_TOK][N4].
template <class T, int NG>
__device__ __forceinline__ void load_group(const void* p, int64_t stride, int64_t row0, int left, int gr, int n, T (&v)[NG]) {
    const char* at = rows_at<T>(p, row0, stride) + (size_t)gr * n * sizeof(T);
    const uint32_t lane = fresh_lane();
#pragma unroll
    for (int e = 0; e < NG; ++e) {
        const uint32_t x = e * 64 + lane;
        v[e] = *reinterpret_cast<const T*>(at + row_off<T>(min((int)(x / Lay<NG>::N4), left - 1), stride, min((int)(x % Lay<NG>::N4), n - 1)));
    }
}
// To LDS in FP32; MASK: zero for padding (from token `live` of the chunk on) and for states that do not exist.
template <bool MASK, class T, int NG>
__device__ __forceinline__ void put_group(const T (&v)[NG], float4* to, int live, int n) {
    const uint32_t lane = fresh_lane();
#pragma unroll
    for (int e = 0; e < NG; ++e) {
        const uint32_t x = e * 64 + lane;
        const bool on = !MASK || ((int)(x / Lay<NG>::N4) < live && (int)(x % Lay<NG>::N4) < n);
        reinterpret_cast<float*>(to)[x] = on ? value_of(v[e]) : 0.0f;
    }
}
// Whether a chunk has no padding, no states and no channels that do not exist: nothing is masked then.
template <int NG>
__device__ __forceinline__ bool whole_chunk(const SsmArgs& a, int tile, int live) {
    return live >= SSM_TOK && a.n == Lay<NG>::N4 && (tile + 1) * Lay<NG>::CH <= a.per;
}

// The decays' factors of a lane's states, times log2 e.
__device__ __forceinline__ void load_rates(const SsmArgs& a, const Place& p, float (&A)[2][4], bool (&okn)[4]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int n = 4 * p.g + s;
        okn[s] = n < a.n;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            A[c][s] = (c ? p.ok1 : p.ok0) && okn[s] ? LOG2E * a.a[(int64_t)(p.c0 + c) * a.n + n] : 0.0f;
    }
}
// Two of a vector's values.
__device__ __forceinline__ float2 load_two(const SsmArgs& a, const float* v, const Place& p) {
    if (!v) return make_float2(0.f, 0.f);
    const int last = p.i + (a.per > 1 ? 1 : 0);
    return make_float2(v[p.odd ? last : p.i], v[last]);
}

// Stands for a segment's decays where a sequence starts in it: nothing crosses that, whatever it was.  Decays too small for FP32 are
// another matter: what is not finite stays so.
constexpr float SEGMENT_STARTS = -1.0f;

// What a segment from nothing leaves: the root of the product of its decays, and its state or cotangent.  The product itself may lie far beyond FP32
// (factors above one are allowed) where the state times it does not; its root is applied twice.
template <int NG>
__device__ __forceinline__ void put_segment(const SsmArgs& a, const Place& p, const float (&A)[2][4], const bool (&okn)[4], float2 total,
                                            bool anew, const float (&h)[2][4]) {
    // the tokens' lanes hold parts of the sum of s
#pragma unroll
    for (int o = 32; o >= Lay<NG>::J; o >>= 1) {
        total.x += __shfl_xor(total.x, o);
        total.y += __shfl_xor(total.y, o);
    }
    char* at = reinterpret_cast<char*>(a.part + ((int64_t)p.b * a.plan.segments + p.seg) * 2 * a.n * a.d);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (!okn[s]) continue;
        const float d0 = anew ? SEGMENT_STARTS : __builtin_amdgcn_exp2f(0.5f * total.x * A[0][s]);
        const float d1 = anew ? SEGMENT_STARTS : __builtin_amdgcn_exp2f(0.5f * total.y * A[1][s]);
        store_pair<float>(at, state_off(a, 4 * p.g + s, p.c0), make_float2(d0, d1), p.ok0, p.ok1);
        store_pair<float>(at, state_off(a, a.n + 4 * p.g + s, p.c0), make_float2(h[0][s], h[1][s]), p.ok0, p.ok1);
    }
}
// A state through a segment.  One that is zero stays so, whatever the decays' product is.
__device__ __forceinline__ float through(float root, float h, float left) {
    return root == SEGMENT_STARTS || h == 0.0f ? left : fmaf(h * root, root, left);
}
// A lane's states h through the segments from, from + step, .. up to `to` (not included), four of them on their way at a time.
__device__ __forceinline__ void through_segments(const SsmArgs& a, const Place& p, int from, int to, int step, float (&h)[2][4]) {
    const int64_t one = (int64_t)2 * a.n * a.d;
    const int count = (to - from) * step;
    uint32_t off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) off[s] = state_off(a, min(4 * p.g + s, a.n - 1), p.i);
    for (int i0 = 0; i0 < count; i0 += 4) {
        Pair<float> decay[4][4], left[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const char* at = reinterpret_cast<const char*>(a.part + ((int64_t)p.b * a.plan.segments + from + step * min(i0 + u, count - 1)) * one);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                decay[u][s] = Pair<float>::load(at, off[s], a.per == 1);
                left[u][s] = Pair<float>::load(at + one * 2, off[s], a.per == 1);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float2 k = own(decay[u][s].get(), p), x = own(left[u][s].get(), p);
                if (i0 + u < count) {
                    h[0][s] = through(k.x, h[0][s], x.x);
                    h[1][s] = through(k.y, h[1][s], x.y);
                }
            }
    }
}

}  // namespace lrs
