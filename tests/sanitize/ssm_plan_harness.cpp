// Walks the selective scan's plan as its launches do, over sizes across the
// accepted range: every chunk of a row lies in one segment, every channel in one
// wave, and no launch has 2^32 threads.  Host arithmetic; no GPU.
#include <stdio.h>
#include <stdlib.h>

#include <cmath>
#include <random>

#include "ssm_plan.hpp"

using namespace lrs;

static void fail(const char* what, long long b, long long l, int d, int n, int g) {
    printf("%s: batch=%lld length=%lld d=%d n=%d groups=%d\n", what, b, l, d, n, g);
    exit(1);
}

static void walk(int64_t b, int64_t l, int d, int n, int g) {
    for (const bool bwd : {false, true}) {
        const SsmPlan p = ssm_plan(b, l, d, n, g, bwd);
        if (p.ng < 2 || p.ng > 16 || p.ng * SSM_STATES < n || (p.ng > 2 && p.ng / 2 * SSM_STATES >= n)) fail("state groups", b, l, d, n, g);
        const int64_t per = d / g, ch = 128 / p.ng;
        if (p.tiles * ch < per || (p.tiles - 1) * ch >= per) fail("tiles", b, l, d, n, g);
        if ((int64_t)p.blocks * p.waves < p.tiles || (int64_t)(p.blocks - 1) * p.waves >= p.tiles) fail("blocks", b, l, d, n, g);
        const int64_t chunks = (l + SSM_TOK - 1) / SSM_TOK;
        if (p.chunks != chunks || p.segments < 1 || p.segments > 64 || p.seg < 1) fail("segments", b, l, d, n, g);
        if ((int64_t)p.segments * p.seg < chunks || (p.segments > 1 && (int64_t)(p.segments - 1) * p.seg >= chunks)) fail("a segment without chunks", b, l, d, n, g);
        const int64_t most = MOST_THREADS / 256;
        if ((bwd ? p.blocks : p.tiles) * (int64_t)g * p.segments * b > most) fail("a launch of too many threads", b, l, d, n, g);
    }
}

int main(int argc, char** argv) {
    const int count = argc > 1 ? atoi(argv[1]) : 1000;
    std::mt19937_64 rng(5);
    const auto spread = [&](double lo, double hi) { return (int64_t)std::llround(std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng))); };
    int walked = 0;
    for (int i = 0; i < count; ++i) {
        const int g = i % 3 ? 1 : (int)spread(1, 64), n = (int)spread(1, 64.4);
        const int d = (int)spread(1, (1 << 21) / g) * g;
        const int64_t b = i % 7 ? spread(1, 1e5) : spread(1, 8), l = i % 5 ? spread(1, 1e5) : spread(1, 2e9);
        if (!ssm_fits(b, l, d, n, g)) continue;
        walk(b, l, d, n, g);
        ++walked;
    }
    if (walked < count / 20) return printf("too few accepted: %d\n", walked), 1;
    for (int64_t l : {0, 1, 15, 16, 17, 1024, 32768})
        for (int d : {1, 2, 31, 32, 33, 2048})
            for (int n : {1, 4, 5, 16, 17, 64}) walk(1, l, d, n, 1);
    if (ssm_shape(1, 1, 0, 1, 1) || ssm_shape(1, 1, 3, 1, 2) || ssm_shape(1, 1, 2, 65, 1) || ssm_shape(2, 1 << 30, 2, 1, 1) || ssm_shape(1, 1, (1 << 21) + 1, 1, 1))
        return printf("an impossible shape is accepted\n"), 1;
    printf("all walked\n");
    return 0;
}
