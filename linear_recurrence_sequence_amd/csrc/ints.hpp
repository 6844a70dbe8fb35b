// ints.hpp -- integer arithmetic shared by host and device code.
#pragma once

#include <stdint.h>

namespace lrs {

constexpr inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace lrs
