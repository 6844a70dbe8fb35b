// lm_ce_plan.hpp -- which tiles, chunks of the vocabulary and ranges of dh's sum
// the linear cross entropy takes for a size.  Host arithmetic only.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "ints.hpp"

namespace lrs {

constexpr int CE_STEP = 64;  // reduction indices of a tile product's step

enum Shape { LARGE, SMALL, FEW };
constexpr int kBM[3] = {256, 128, 64}, kBN[3] = {256, 128, 32};

// Tokens up to which the backward goes by the bytes of w and dw: dz lies [entries, tokens], and dw is streamed.  By that and by the
// form for many tokens, 2048 x 128000: 33 tokens 412 and 471 us, 128 466 and 523, 129 595 and 564, 192 598 and 610, 256 607 and 648;
// 1024 x 32000: 64 60 and 70, 129 90 and 98, 256 98 and 104.  Small heads gain nothing from it: 512 x 4000, 256 tokens, 38 and 33.
constexpr int kFew = 256;
constexpr int64_t kMostDz = (int64_t)128 << 20;  // elements of dz held at once

// Time of a product of p x q results over k, in microseconds: rounds of
// workgroups, each its steps of 64 and the start and end of a tile.  A large tile's step
// takes 1.45 us and its start and end 6; two small ones of a CU 1.0 and 5, and one
// alone 0.7 (measured over long and short k with the CUs busy).
inline double product_us(Shape s, int64_t p, int64_t q, int64_t k) {
    const int64_t tiles = ceil_div(p, kBM[s]) * ceil_div(q, kBN[s]);
    const double steps = (double)ceil_div(k, CE_STEP);
    if (s == LARGE) return (double)ceil_div(tiles, 256) * (steps * 1.45 + 6.0);
    const int64_t rest = tiles % 512;
    return (double)(tiles / 512) * (steps + 5.0) + (rest == 0 ? 0.0 : rest <= 256 ? steps * 0.7 + 5.0 : steps + 5.0);
}

// How many of `rows` vocabulary entries go by large tiles, against `other` rows
// over k: all, none, or the whole rounds of them, the rest then going by small
// tiles in a launch of its own (486 x 2384 x 33847 is 266 large tiles, ten more than a
// round).  A multiple of 256, or all.
inline int64_t large_rows(int64_t rows, int64_t other, int64_t k, double* us = nullptr) {
    const int64_t across = ceil_div(other, 256), whole = ceil_div(rows, 256) * across / 256 * 256 / across * 256;
    int64_t best = 0;
    double least = product_us(SMALL, rows, other, k);
    for (int64_t large : {rows, whole}) {
        if (large <= 0 || large > rows) continue;
        // two launches have to be worth a tenth
        const double t = large == rows ? product_us(LARGE, rows, other, k)
                                       : 1.1 * (product_us(LARGE, large, other, k) + product_us(SMALL, rows - large, other, k) + 3.0);
        if (t <= least) least = t, best = large;
    }
    if (us) *us = least;
    return best;
}

inline int ce_parts(int n, int d, int v) {
    if (n <= 32) return (int)ceil_div(v, kBM[FEW]);
    const int64_t large = large_rows(v, n, d);
    return (int)(ceil_div(large, 256) + ceil_div(v - large, 128));
}

// Vocabulary entries that one launch of a shape's tiles takes against n tokens, a whole number of tiles.
inline int64_t ce_launch_rows(Shape s, int threads, int64_t n) { return MOST_THREADS / threads / ceil_div(n, kBN[s]) * kBM[s]; }

// Sizes that are taken.  Indices are 31 bits, tiles included; the launches over tokens take up to 64 threads
// a token, and the one that joins dh a thread for four of its elements.
inline bool ce_shape(int64_t n, int d, int64_t v) {
    return n >= 0 && n <= (1 << 26) - 16 && v >= 1 && v < 0x7fffffff - 512 && d >= 8 && d <= 65536 && d % 8 == 0 &&
           n * d <= 4 * (MOST_THREADS - 255) && ceil_div(n, 128) * ceil_div(v, 128) < 0x7fffffff;
}

struct CePlan {
    int chunk;   // vocabulary entries a backward pass takes at a time (a multiple of 256)
    int splits;  // ranges of a chunk summed apart for dh, at most
    int range;   // entries of a range, a whole number of steps
    int dh;      // tile shape of its product
    int few;     // columns of a transposed dz (32, 64, 128 or 256), 0 with many tokens
};

// The range that cuts a chunk of `count` entries into about `splits`, and how many it makes.  It is formed once, from the
// first chunk, which is the longest, and holds for all: rounding to whole steps is not monotone, so that a range of its own could cut a
// shorter chunk into more pieces than the workspace holds and the last launch sums.
inline void ce_set_range(CePlan& p, int64_t count) {
    p.range = (int)(ceil_div(ceil_div(count, p.splits), CE_STEP) * CE_STEP);
    p.splits = (int)ceil_div(count, p.range);
}

// Chunks of the vocabulary, tiles and the ranges that dh is summed over: the
// cheapest by product_us and the bytes of dh's partial sums, over the chunk
// counts from the least that the buffer of dz allows.
inline CePlan ce_plan(int n, int d, int v) {
    n = std::max(n, 1);
    if (n <= kFew) {
        CePlan p{};
        p.few = n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256;
        const int64_t chunks = ceil_div(v, kMostDz / p.few / 256 * 256);
        p.chunk = (int)(ceil_div(ceil_div(v, chunks), 256) * 256);
        p.dh = n <= 32 ? FEW : SMALL;
        // the product over the vocabulary reads w once: enough ranges to fill the chip, four steps or more each
        const int64_t tiles = ceil_div(d, kBM[p.dh]) * ceil_div(n, kBN[p.dh]), want = (p.dh == FEW ? 1024 : 512) / tiles;
        p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(want, std::min(p.chunk, v) / (4 * CE_STEP)));
        ce_set_range(p, std::min(p.chunk, v));
        return p;
    }
    const int64_t most = std::max<int64_t>(256, kMostDz / n / 256 * 256), least = ceil_div(v, most);
    CePlan best{};
    double best_us = 0.0;
    for (int64_t chunks = least; chunks < least + 8; ++chunks) {
        const int64_t chunk = ceil_div(ceil_div(v, chunks), 256) * 256, count = std::min<int64_t>(chunk, v);
        CePlan p{};
        p.chunk = (int)chunk;
        double us, dw_us, dh_us = 0.0;
        large_rows(count, n, d, &us);
        large_rows(count, d, n, &dw_us);
        us += dw_us;
        for (int s = LARGE; s <= SMALL; ++s) {
            for (int splits = 1; splits <= 64 && (splits == 1 || count / splits >= 8 * CE_STEP); ++splits) {
                // the partial sums are written, and read by the next chunk or the last launch
                const double t = product_us((Shape)s, d, ceil_div(n, kBN[s]) * kBN[s] * splits, ceil_div(count, splits)) + (double)splits * n * d * 8 / 4.5e6;
                if (dh_us == 0.0 || t < dh_us) dh_us = t, p.dh = s, p.splits = splits;
            }
        }
        us = (us + dh_us) * (double)ceil_div(v, chunk);
        if (best_us == 0.0 || us < best_us) best_us = us, best = p;
    }
    ce_set_range(best, std::min(best.chunk, v));
    return best;
}

// Chunk i of the vocabulary: its first entry, its entries, and the ranges that dh's sum over it is cut into.
struct CeChunk {
    int first, count, splits;
};
inline int ce_chunks(const CePlan& p, int v) { return (int)ceil_div(v, p.chunk); }
inline CeChunk ce_chunk(const CePlan& p, int v, int i) {
    const int64_t first = (int64_t)i * p.chunk, count = std::min<int64_t>(p.chunk, v - first);  // first + chunk may pass 2^31
    return {(int)first, (int)count, (int)ceil_div(count, p.range)};
}

}  // namespace lrs
