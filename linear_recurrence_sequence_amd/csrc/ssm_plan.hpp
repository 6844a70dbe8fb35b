// ssm_plan.hpp -- how the selective scan is spread over the chip.  Plain host
// code, shared by the launches and the workspace sizes.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "ints.hpp"

namespace lrs {

constexpr int SSM_TOK = 16;       // tokens of a chunk: a state is kept before each
constexpr int SSM_STATES = 4;     // states of a lane, for two channels
constexpr int SSM_MOST_N = 64;
constexpr int64_t SSM_MOST_STRIDE = (1 << 22) - 1;  // a chunk's rows are addressed by 24-bit products and 32-bit offsets

// A wave takes 128 / ng channels and all states: its lanes are ng groups (of
// SSM_STATES states each) of 64 / ng channel pairs.  Two groups at least: up to four states on one group take 80 and 249 us
// forward and backward (2 x 2048 x 2048, BF16), five on two groups 75 and 172.
inline int ssm_state_groups(int n) {
    int ng = 2;
    while (ng * SSM_STATES < n) ng *= 2;
    return ng;
}

struct SsmPlan {
    int ng;               // state groups of a wave
    int tiles;            // waves over the channels of one group of b and c
    int waves;            // waves of a workgroup (in the backward they share one group of b and c)
    int blocks;           // backward: workgroups over the channels of one group of b and c
    int chunks;           // of a row
    int segments, seg;    // parts of a row worked on at once, chunks of each
};

// The recurrence runs through a row.  Rows and channels alone are too few waves where a batch is small, so a row
// is cut into segments: each is first run from a zero state (half of the work again), then from the state that the
// segments before it leave.  Waves a SIMD, and microseconds of both launches, 16 states, BF16 with a gate:
//                            1          2          3          4          6
//   4 x 1024 x 2048          45 + 80    36 + 54    38 + 56    35 + 61    39 + 65
//   2 x 2048 x 2048          45 + 89    36 + 60    39 + 59    35 + 71    39 + 82
//   1 x 32768 x 2048         330 + 644  260 + 383  249 + 362  241 + 372  240 + 368
// More waves hide more, until each walks so few tokens that going through the segments before it (one state read for
// each) costs more: three where that leaves 256 tokens or more to each, else two.  In the backward two: 2 x 2048 x 2048 with one, two and four
// 47 + 248, 40 + 173 and 39 + 187.  All of this was timed with 16 states.  Of these, three waves of the gated scan fit a SIMD at once and two
// of the backward; up to 8 states two (FP32) or three and one, 17 to 32 two and two, 33 to 64 one and one.  The same plan serves them.
// 64 segments are the most, so that a narrow row leaves SIMDs idle: 1 x 32768 takes 224 + 535 us at a width of 64, 243 + 541 at 512 and 529 + 1313
// at 2048 (forward with the states kept, and backward).
constexpr int64_t SIMDS = 1024;

inline SsmPlan ssm_plan(int64_t batch, int64_t length, int d, int n, int groups, bool backward) {
    SsmPlan p{};
    p.ng = ssm_state_groups(n);
    p.waves = 4;
    p.tiles = (int)ceil_div(d / groups, 128 / p.ng);
    p.blocks = (int)ceil_div(p.tiles, p.waves);
    p.chunks = (int)ceil_div(length, SSM_TOK);
    const int64_t units = std::max<int64_t>(1, batch * groups * (backward ? (int64_t)p.blocks * p.waves : p.tiles));
    const int64_t want = SIMDS * (!backward && p.chunks / std::max<int64_t>(1, 3 * SIMDS / units) >= 256 / SSM_TOK ? 3 : 2);
    const int64_t s = std::max<int64_t>(1, std::min<int64_t>({want / units, 64, p.chunks}));
    p.seg = (int)ceil_div(std::max(1, p.chunks), s);
    p.segments = (int)ceil_div(std::max(1, p.chunks), p.seg);
    return p;
}

inline bool ssm_shape(int64_t batch, int64_t length, int d, int n, int groups) {
    return batch >= 0 && length >= 0 && length <= 0x7fffff00 && batch <= 0x7fffffff && (length == 0 || batch <= 0x7fffffff / length) &&
           d >= 1 && d <= (1 << 21) && groups >= 1 && d % groups == 0 && n >= 1 && n <= SSM_MOST_N;
}

// The backward's last launch: workgroups of 256 sums, first of db and dc (two values for each row, group and padded state), then of da, dskip and
// ddt_bias (n + 2 for each channel).  Together they may need more threads than a launch has: then there are several, of `grid` workgroups at most.
struct SsmJoin {
    int64_t narrow, all;  // workgroups of db and dc, and of everything
    unsigned grid;
};
inline SsmJoin ssm_join(int64_t batch, int64_t length, int d, int n, int groups, int ng) {
    SsmJoin j{};
    j.narrow = ceil_div(batch * length * groups * 2 * SSM_STATES * ng, 256);
    j.all = j.narrow + ceil_div((int64_t)d * (n + 2), 256);
    j.grid = (unsigned)std::min<int64_t>(j.all, MOST_THREADS / 256);
    return j;
}

// Sizes that the launches cover: fewer than 2^24 waves forward and workgroups of 256 backward (the step has 16 threads a channel at most, which is
// fewer; the last launch takes any number), and element counts within 62 bits.
inline bool ssm_fits(int64_t batch, int64_t length, int d, int n, int groups) {
    if (!ssm_shape(batch, length, d, n, groups)) return false;
    const int64_t chunks = ceil_div(std::max<int64_t>(length, 1), SSM_TOK), most = MOST_THREADS / 256;
    const SsmPlan f = ssm_plan(batch, length, d, n, groups, false), b = ssm_plan(batch, length, d, n, groups, true);
    const __int128 state = (__int128)batch * chunks * d * SSM_MOST_N * 4, rows = (__int128)batch * length * groups;
    return (__int128)batch * groups * f.tiles * f.segments <= most && (__int128)batch * groups * b.blocks * b.segments <= most &&
           state < ((__int128)1 << 62) && rows * b.blocks * SSM_MOST_N * 8 < ((__int128)1 << 62);
}

}  // namespace lrs
