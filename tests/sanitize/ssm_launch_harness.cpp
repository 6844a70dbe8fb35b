// The backward's last launch of the selective scan at the widest accepted sizes:
// fewer than 2^32 threads, and every sum of db, dc, da, dskip and ddt_bias belongs to
// one workgroup that the grid reaches.  Host arithmetic; no GPU.
#include <stdio.h>
#include <stdlib.h>

#include <cmath>
#include <random>

#include "ssm_plan.hpp"

using namespace lrs;

static int seen = 0;

static void check(int64_t b, int64_t l, int d, int n, int g) {
    if (!ssm_fits(b, l, d, n, g)) return;
    ++seen;
    const int ng = ssm_plan(b, l, d, n, g, true).ng;
    const SsmJoin j = ssm_join(b, l, d, n, g, ng);
    const __int128 narrow = (__int128)b * l * g * 2 * SSM_STATES * ng, wide = (__int128)d * (n + 2);
    const bool ok = j.grid >= 1 && (int64_t)j.grid * 256 <= MOST_THREADS && (__int128)j.narrow * 256 >= narrow && (__int128)(j.all - j.narrow) * 256 >= wide &&
                    (__int128)j.narrow * 256 < narrow + 256 && j.all >= j.grid;
    if (!ok) {
        printf("the last launch: batch=%lld length=%lld d=%d n=%d groups=%d\n", (long long)b, (long long)l, d, n, g);
        exit(1);
    }
}

int main() {
    // where the two parts together pass 2^32 threads
    for (int n : {1, 8, 9, 16, 17, 32, 33, 64})
        for (int d : {1, 64, 512})
            for (int64_t rows = (1 << 25) - 300; rows < (1 << 25) + 300; ++rows) check(1, rows, d, n, 1), check(rows, 1, d, n, 1);
    std::mt19937_64 rng(7);
    const auto spread = [&](double lo, double hi) { return (int64_t)std::llround(std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng))); };
    for (int i = 0; i < 100000; ++i) {
        const int g = i % 3 ? 1 : (int)spread(1, 64);
        check(spread(1, 1e5), spread(1, 2e9), (int)spread(1, (1 << 21) / g) * g, (int)spread(1, 64.4), g);
    }
    if (seen < 10000) return printf("too few accepted: %d\n", seen), 1;
    printf("all covered\n");
    return 0;
}
