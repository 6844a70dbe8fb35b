// ints.hpp -- integer arithmetic shared by host and device code.
#pragma once

#include <stdint.h>

namespace lrs {

constexpr inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch's threads along x are 32 bits: of more, the runtime runs what is left modulo 2^32, without an error.
constexpr int64_t MOST_THREADS = 0xffffffffll;

}  // namespace lrs
