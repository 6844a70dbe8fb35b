// ssm_lay.hpp -- where a wave of the selective scan stands, and how it reads a
// chunk.
#pragma once

#include "ssm.hpp"

namespace lrs {

template <int NG>
struct Lay {
    static constexpr int J = 64 / NG, CH = 2 * J, N4 = SSM_STATES * NG, Q = SSM_TOK / NG;
};

// A wave's row and segment, its lane's channels.
struct Place {
    int b, seg, gr, c0, end;     // row, segment, group of b and c, the lane's first channel, the group's end
    int i, k;                    // channels that the lane loads: its own, or existing ones in their place
    bool ok0, ok1, pair;
};
template <int NG>
__device__ __forceinline__ Place place_of(const SsmArgs& a, int tile, int gr, int seg, int b) {
    const int j = (threadIdx.x & 63) % Lay<NG>::J;
    Place p;
    p.b = b, p.seg = seg, p.gr = gr;
    p.end = (gr + 1) * a.per;
    p.c0 = gr * a.per + tile * Lay<NG>::CH + 2 * j;
    p.ok0 = p.c0 < p.end, p.ok1 = p.c0 + 1 < p.end;
    p.pair = a.per % 2 == 0;
    p.i = min(p.c0, p.end - (p.pair ? 2 : 1));
    p.k = min(p.c0 + 1, p.end - 1);
    return p;
}

__device__ __forceinline__ int length_of(const SsmArgs& a, int b) {
    return a.lengths ? min(max(a.lengths[b], 0), a.length) : a.length;
}

// Bit t: token t0 + t of row b starts a sequence.
__device__ __forceinline__ uint32_t resets_of(const SsmArgs& a, int b, int t0, int len) {
    if (!a.reset) return 0u;
    const int t = t0 + (threadIdx.x & 63);
    const bool r = t < min(t0 + SSM_TOK, len) && a.reset[(int64_t)b * a.length + t] != 0;
    return (uint32_t)__ballot(r);
}

}  // namespace lrs
