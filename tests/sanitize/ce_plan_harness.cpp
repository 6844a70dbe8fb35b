// Walks the linear cross entropy's plan as its launches do, over sizes across
// the whole accepted range: what a chunk of the vocabulary writes has to be what
// the last launch sums, inside the workspace.  Host arithmetic; no GPU.
#include <stdio.h>
#include <stdlib.h>

#include <cmath>
#include <random>

#include "lm_ce_plan.hpp"

using namespace lrs;

static long long several, worst_chunks;

static void fail(const char* what, int n, int d, int v) {
    printf("%s: n=%d d=%d v=%d\n", what, n, d, v);
    exit(1);
}

// Every launch's threads, and the parts that the forward's launches number.
static void launches(int n, int d, int v, const CePlan& p) {
    const auto threads = [&](int64_t tiles, int each) {
        if (tiles < 1 || tiles * each > MOST_THREADS) fail("a launch of too many threads", n, d, v);
    };
    const int large = n <= 32 ? 0 : (int)large_rows(v, n, d);
    int64_t part = 0;
    for (int64_t v0 = 0; v0 < v;) {
        const Shape s = n <= 32 ? FEW : v0 < large ? LARGE : SMALL;
        const int each = s == LARGE ? 512 : 256;
        const int64_t some = std::min<int64_t>((s == LARGE ? large : v) - v0, ce_launch_rows(s, each, n));
        if (some < 1) fail("a launch without rows", n, d, v);
        if (some % kBM[s] && v0 + some != (s == LARGE ? large : v)) fail("a launch cut inside a tile", n, d, v);
        threads(ceil_div(some, kBM[s]) * ceil_div(n, kBN[s]), each);
        part += ceil_div(some, kBM[s]);
        v0 += some;
    }
    if (part != ce_parts(n, d, v)) fail("parts", n, d, v);
    threads(ceil_div(n, 16), 1024);
    threads(ceil_div(n, 4), 256);
    const CeChunk c = ce_chunk(p, v, 0);
    const int64_t quads = (int64_t)n * d / 4;
    for (int s : {LARGE, SMALL, FEW}) {
        if ((s == FEW) != (n <= 32)) continue;
        threads(ceil_div(c.count, kBM[s]) * ceil_div(p.few ? p.few : n, kBN[s]), s == LARGE ? 512 : 256);
        if (!p.few) threads(ceil_div(d, kBM[s]) * ceil_div(c.count, kBN[s]), 256);
    }
    threads(ceil_div(d, kBM[p.dh]) * ceil_div(n, kBN[p.dh]) * p.splits, 256);
    threads(p.splits >= 16 ? ceil_div(quads, 32) : ceil_div(quads, 256), 256);
}

static void walk(int n, int d, int v) {
    if (!ce_shape(n, d, v)) return;
    const CePlan p = ce_plan(n, d, v);
    if (p.chunk < 256 || p.chunk % 256 || p.splits < 1 || (p.few ? n > p.few : n <= 256)) fail("plan", n, d, v);
    const int chunks = ce_chunks(p, v);
    int64_t next = 0;
    for (int i = 0; i < chunks; ++i) {
        // of very many chunks the first and the last ones
        if (i == 1000 && chunks > 2000) next = (int64_t)p.chunk * (i = chunks - 1000);
        const CeChunk c = ce_chunk(p, v, i);
        if (c.first != next || c.count < 1 || c.count > p.chunk) fail("chunks do not follow each other", n, d, v);
        next += c.count;
        if (p.range < CE_STEP || p.range % CE_STEP || c.splits < 1) fail("range", n, d, v);
        if ((int64_t)p.range * c.splits < c.count || (int64_t)p.range * (c.splits - 1) >= c.count) fail("ranges do not cover the chunk", n, d, v);
        if (c.splits > p.splits) fail("a chunk has more ranges than are summed", n, d, v);
    }
    if (next != v) fail("chunks do not cover the vocabulary", n, d, v);
    launches(n, d, v, p);
    several += chunks > 1;
    worst_chunks = std::max<long long>(worst_chunks, chunks);
}

int main(int argc, char** argv) {
    const int rounds = argc > 1 ? atoi(argv[1]) : 10000;
    const int seen[][3] = {{141, 72, 557087}, {206, 304, 674427}, {80, 400, 2605384}, {200, 64, 589826}, {247, 200, 589971}, {91, 264, 1066594},
                           {1, 8, 1}, {32, 8, 0x7fffffff - 513}, {256, 65536, 0x7fffffff - 513}, {257, 8, 1 << 22}, {700000, 8, 0x7fffffff - 513},
                           {(1 << 26) - 16, 8, 300}, {(1 << 26) - 16, 256, 1}, {262143, 65528, 1000}, {1 << 22, 4088, 131072}, {40, 8, 0x7fffffff - 513}, {8192, 2048, 128000}};
    for (const auto& s : seen) walk(s[0], s[1], s[2]);
    std::mt19937_64 rng(1);
    const auto spread = [&](double lo, double hi) { return (int)std::exp(std::uniform_real_distribution<>(std::log(lo), std::log(hi))(rng)); };
    for (int i = 0; i < rounds; ++i) {
        walk(spread(1, 257), 8 * spread(1, 1024), spread(3e5, 2e7));   // few tokens, about one chunk and more
        walk(spread(129, 257), 8 * spread(1, 64), spread(5e5, 3e6));
        walk(spread(257, 20000), 8 * spread(1, 1024), spread(1, 1e6));
        walk(spread(1, 20000), 8 * spread(1, 64), spread(1, 4e6));
        walk(spread(1, 6e7), 8 * spread(1, 8192), spread(1, 2e9));
    }
    printf("%lld of several chunks, at most %lld; all walked\n", several, worst_chunks);
    return 0;
}
