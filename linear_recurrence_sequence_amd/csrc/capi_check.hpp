// capi_check.hpp -- argument checks shared by the C ABI files.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>
#include <string>

#include "internal.hpp"
#include "samu_scan.h"

namespace lrs {
namespace {

scan_status fail(scan_status st, const std::string& msg) { return (scan_status)set_last_error(st, msg.c_str()); }

// A tensor argument: `n` bytes from p, aligned to `align` bytes.
struct Arg {
    const void* p;
    size_t n, align;
    const char* name;
};

scan_status check_args(std::initializer_list<Arg> req, std::initializer_list<Arg> opt) {
    for (const Arg& a : req)
        if (!a.p) return fail(SCAN_ERR_NULL, std::string(a.name) + " is NULL");
    for (const auto* list : {&req, &opt})
        for (const Arg& a : *list)
            if (a.p && ((uintptr_t)a.p & (a.align - 1)))
                return fail(SCAN_ERR_ALIGN, std::string(a.name) + " is not " + std::to_string(a.align) + "-byte aligned");
    return SCAN_OK;
}

bool overlap(const Arg& a, const Arg& b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// outputs must not overlap inputs nor each other
scan_status check_alias(std::initializer_list<Arg> ins, std::initializer_list<Arg> outs) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Arg& i : ins)
            if (overlap(*o, i)) return fail(SCAN_ERR_ALIAS, std::string(o->name) + " overlaps " + i.name);
        for (auto q = o + 1; q != outs.end(); ++q)
            if (overlap(*o, *q)) return fail(SCAN_ERR_ALIAS, std::string(o->name) + " overlaps " + q->name);
    }
    return SCAN_OK;
}

scan_status device_status(hipError_t e, const char* where) {
    if (e == hipSuccess) return SCAN_OK;
    return fail(SCAN_ERR_DEVICE, std::string(where) + ": " + hipGetErrorString(e));
}

bool dtype_ok(int t) { return t == SCAN_BF16 || t == SCAN_F32; }
size_t dtype_size(int t) { return t == SCAN_F32 ? 4 : 2; }
// bytes from the first to the last element of `rows` rows
size_t span(int64_t rows, int64_t stride, int d, size_t size) {
    return rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)d) * size : 0;
}

}  // namespace
}  // namespace lrs
