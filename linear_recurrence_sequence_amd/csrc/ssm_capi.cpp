// ssm_capi.cpp -- the C ABI of the selective state space mixer (ssm_ops.h):
// argument validation, workspace layout and kernel sequencing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "capi_check.hpp"
#include "ssm.hpp"
#include "ssm_ops.h"

namespace lrs {
namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;
static_assert(SSM_CHUNK == SSM_TOK && SSM_MAX_STATE == SSM_MOST_N, "the header's limits");

scan_status check_strides(const char* fn, std::initializer_list<int64_t> strides, int64_t most = kMaxStride) {
    for (int64_t s : strides)
        if (s < 0 || s > most) return fail(SCAN_ERR_SHAPE, std::string(fn) + ": row strides must lie in 0.." + std::to_string(most));
    return SCAN_OK;
}

scan_status ssm_check(const char* fn, int64_t batch, int64_t length, int d, int n, int groups, int dtype,
                      std::initializer_list<int64_t> strides, int64_t most_stride) {
    if (!ssm_fits(batch, length, d, n, groups))
        return fail(SCAN_ERR_SHAPE, std::string(fn) + ": unsupported shape batch=" + std::to_string(batch) + " length=" + std::to_string(length) +
                                        " d=" + std::to_string(d) + " n=" + std::to_string(n) + " groups=" + std::to_string(groups) +
                                        " (need d a multiple of groups, 1 <= n <= " + std::to_string(SSM_MAX_STATE) +
                                        ", d <= 2^21, batch * length < 2^31 and fewer than 2^24 waves, one for each row and 128 / g channels of a group: g = 2, 4, 8, 16 for n up "
                                        "to 8, 16, 32, 64)");
    if (!dtype_ok(dtype)) return fail(SCAN_ERR_SHAPE, std::string(fn) + ": dtype must be SCAN_BF16 or SCAN_F32");
    return check_strides(fn, strides, most_stride);
}

scan_status check_workspace(const char* fn, size_t have, size_t need) {
    if (have >= need) return SCAN_OK;
    return fail(SCAN_ERR_WORKSPACE, std::string(fn) + ": workspace_bytes " + std::to_string(have) + " < " + std::to_string(need));
}

size_t ssm_layout(bool bwd, int64_t batch, int64_t length, int d, int n, int groups, void* base, SsmArgs* a) {
    char* p = static_cast<char*>(base);
    size_t off = 0;
    const auto take = [&](size_t floats) {
        float* at = reinterpret_cast<float*>(p ? p + off : nullptr);
        off += (floats * 4 + 255) / 256 * 256;
        return at;
    };
    const SsmPlan pl = ssm_plan(batch, length, d, n, groups, bwd);
    const size_t parts = (size_t)batch * pl.segments;
    a->plan = pl;
    a->part = take(pl.segments > 1 ? parts * 2 * n * d : 0);
    if (bwd) {
        a->part_bc = take((size_t)groups * pl.blocks * batch * length * 2 * SSM_STATES * pl.ng);
        a->part_a = take(parts * n * d);
        a->part_d = take(parts * 2 * d);
    }
    return std::max<size_t>(off, 256);
}

bool conv_shape(int64_t batch, int64_t length, int d, int width) {
    return batch >= 0 && length >= 0 && length <= 0x7fffff00 && batch <= 0x7fffffff && (length == 0 || batch <= 0x7fffffff / length) && d >= 1 &&
           d <= (1 << 24) && width >= 2 && width <= CONV_MAX_WIDTH;
}

// Tokens of a piece of a row.  A piece reads width - 1 tokens again on either side, and in the backward leaves its sums for the
// weights' gradients: half as many pieces there.  2 x 2048 x 2048 in BF16, pieces of 8, 16, 32 and 64 tokens: forward 11.4, 12.4, 14.0 and
// 22 us, backward with the sums 37, 27, 27 and 36; 32768 x 2560, 16 to 128 tokens: 92, 85, 84 and 118, backward 288, 229, 212 and 246.
void conv_plan(int64_t batch, int64_t length, int d, bool backward, ConvArgs* a) {
    const int64_t quads = ceil_div(d, 4), want = std::max<int64_t>(1, (1 << (backward ? 17 : 18)) / std::max<int64_t>(1, quads * batch));
    const int64_t tokens = ceil_div(std::max<int64_t>(length, 1), want);
    a->tokens = (int)std::min<int64_t>(64, ceil_div(std::max<int64_t>(tokens, 8), 8) * 8);
    a->pieces = (int)std::max<int64_t>(1, ceil_div(length, a->tokens));
}
bool conv_fits(int64_t batch, int64_t length, int d, int width) {
    if (!conv_shape(batch, length, d, width)) return false;
    ConvArgs a{};
    conv_plan(batch, length, d, false, &a);
    return (__int128)batch * a.pieces * ceil_div(d, 2) <= MOST_THREADS - 256;
}
size_t conv_part_bytes(int64_t batch, int64_t length, int d, int width) {
    ConvArgs a{};
    conv_plan(batch, length, d, true, &a);
    return std::max<size_t>(256, (size_t)batch * a.pieces * (width + 1) * d * 4);
}
scan_status conv_check(const char* fn, int64_t batch, int64_t length, int d, int width, int dtype, int act, std::initializer_list<int64_t> strides) {
    if (!conv_fits(batch, length, d, width))
        return fail(SCAN_ERR_SHAPE, std::string(fn) + ": unsupported shape batch=" + std::to_string(batch) + " length=" + std::to_string(length) +
                                        " d=" + std::to_string(d) + " width=" + std::to_string(width) + " (need 1 <= d <= 2^24, 2 <= width <= " +
                                        std::to_string(CONV_MAX_WIDTH) + ", batch * length < 2^31 and a launch below 2^32 threads)");
    if (!dtype_ok(dtype)) return fail(SCAN_ERR_SHAPE, std::string(fn) + ": dtype must be SCAN_BF16 or SCAN_F32");
    if (act != CONV_NONE && act != CONV_SILU) return fail(SCAN_ERR_SHAPE, std::string(fn) + ": act must be CONV_NONE or CONV_SILU");
    return check_strides(fn, strides);
}

}  // namespace
}  // namespace lrs

using namespace lrs;

extern "C" {

// ------------------------------------------------------ selective scan ---
size_t ssm_scan_saved_bytes(int64_t batch, int64_t length, int d, int n, int groups) {
    if (!ssm_fits(batch, length, d, n, groups)) return 0;
    return std::max<size_t>(256, (size_t)batch * ceil_div(length, SSM_TOK) * n * d * 4);
}

size_t ssm_scan_workspace_bytes(int64_t batch, int64_t length, int d, int n, int groups, int backward) {
    if (!ssm_fits(batch, length, d, n, groups)) return 0;
    SsmArgs a{};
    return ssm_layout(backward != 0, batch, length, d, n, groups, nullptr, &a);
}

scan_status ssm_scan_fwd(int64_t batch, int64_t length, int d, int n, int groups, int dtype, int softplus, const void* u, int64_t u_stride,
                         const void* dt, int64_t dt_stride, const float* a, const void* b, int64_t b_stride, const void* c, int64_t c_stride,
                         const float* skip, const void* z, int64_t z_stride, const float* dt_bias, const float* h0, const uint8_t* reset,
                         const int32_t* lengths, void* y, float* h_final, void* saved, void* workspace, size_t workspace_bytes, void* stream) {
    scan_status st = ssm_check("ssm_scan_fwd", batch, length, d, n, groups, dtype, {u_stride, dt_stride, b_stride, c_stride, z_stride}, SSM_MOST_STRIDE);
    if (st != SCAN_OK) return st;
    if (batch == 0) return SCAN_OK;
    const size_t es = dtype_size(dtype), state = (size_t)batch * d * n * 4;
    const int64_t rows = batch * length;
    SsmArgs k{};
    const size_t need = ssm_layout(false, batch, length, d, n, groups, nullptr, &k);
    const auto some = [&](const void* p) { return length > 0 ? p : nullptr; };
    const Arg au{some(u), span(rows, u_stride, d, es), es, "u"}, at{some(dt), span(rows, dt_stride, d, es), es, "dt"},
        aa{a, (size_t)d * n * 4, 4, "a"}, ab{some(b), span(rows, b_stride, groups * n, es), es, "b"},
        ac{some(c), span(rows, c_stride, groups * n, es), es, "c"}, as{skip, (size_t)d * 4, 4, "skip"},
        az{some(z), span(rows, z_stride, d, es), es, "z"}, ai{dt_bias, (size_t)d * 4, 4, "dt_bias"}, ah{h0, state, 4, "h0"},
        ar{some(reset), (size_t)rows, 1, "reset"}, al{lengths, (size_t)batch * 4, 4, "lengths"}, oy{some(y), (size_t)rows * d * es, es, "y"},
        oh{h_final, state, 4, "h_final"}, os{some(saved), ssm_scan_saved_bytes(batch, length, d, n, groups), 16, "saved"},
        ws{workspace, need, 16, "workspace"};
    st = length > 0 ? check_args({au, at, aa, ab, ac, oy, oh, ws}, {as, az, ai, ah, ar, al, os}) : check_args({aa, oh, ws}, {as, ai, ah, al});
    if (st == SCAN_OK) st = check_workspace("ssm_scan_fwd", workspace_bytes, need);
    if (st == SCAN_OK) st = check_alias({au, at, aa, ab, ac, as, az, ai, ah, ar, al}, {oy, oh, os, ws});
    if (st != SCAN_OK) return st;
    ssm_layout(false, batch, length, d, n, groups, workspace, &k);
    k.batch = (int)batch, k.length = (int)length, k.d = d, k.n = n, k.groups = groups, k.per = d / groups, k.softplus = softplus != 0;
    k.u = u, k.dt = dt, k.b = b, k.c = c, k.z = z;
    k.u_stride = u_stride, k.dt_stride = dt_stride, k.b_stride = b_stride, k.c_stride = c_stride, k.z_stride = z_stride;
    k.a = a, k.skip = skip, k.dt_bias = dt_bias, k.h0 = h0, k.reset = reset, k.lengths = lengths;
    k.y = y, k.h = h_final, k.saved = static_cast<float*>(saved);
    return device_status(launch_ssm_fwd(k, dtype == SCAN_F32, (hipStream_t)stream), "selective scan");
}

scan_status ssm_scan_bwd(int64_t batch, int64_t length, int d, int n, int groups, int dtype, int softplus, const void* u, int64_t u_stride,
                         const void* dt, int64_t dt_stride, const float* a, const void* b, int64_t b_stride, const void* c, int64_t c_stride,
                         const float* skip, const void* z, int64_t z_stride, const float* dt_bias, const uint8_t* reset, const int32_t* lengths,
                         const void* saved, const void* dy, int64_t dy_stride, const float* dh_final, void* du, void* ddt, float* da, void* db,
                         void* dc, float* dskip, void* dz, float* ddt_bias, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    scan_status st = ssm_check("ssm_scan_bwd", batch, length, d, n, groups, dtype, {u_stride, dt_stride, b_stride, c_stride, z_stride, dy_stride},
                               SSM_MOST_STRIDE);
    if (st != SCAN_OK) return st;
    const size_t es = dtype_size(dtype), state = (size_t)batch * d * n * 4;
    const int64_t rows = batch * length;
    if (rows > 0 && z && !dz) return fail(SCAN_ERR_NULL, "dz is NULL");
    SsmArgs k{};
    const size_t need = ssm_layout(true, batch, length, d, n, groups, nullptr, &k), wide = (size_t)rows * d * es,
                 narrow = (size_t)rows * groups * n * es;
    const auto some = [&](const void* p) { return rows > 0 ? p : nullptr; };
    const Arg au{some(u), span(rows, u_stride, d, es), es, "u"}, at{some(dt), span(rows, dt_stride, d, es), es, "dt"},
        aa{a, (size_t)d * n * 4, 4, "a"}, ab{some(b), span(rows, b_stride, groups * n, es), es, "b"},
        ac{some(c), span(rows, c_stride, groups * n, es), es, "c"}, as{skip, (size_t)d * 4, 4, "skip"},
        az{some(z), span(rows, z_stride, d, es), es, "z"}, ai{dt_bias, (size_t)d * 4, 4, "dt_bias"}, ar{some(reset), (size_t)rows, 1, "reset"},
        al{lengths, (size_t)batch * 4, 4, "lengths"}, av{some(saved), ssm_scan_saved_bytes(batch, length, d, n, groups), 16, "saved"},
        ay{some(dy), span(rows, dy_stride, d, es), es, "dy"}, ah{dh_final, state, 4, "dh_final"}, ou{some(du), wide, es, "du"},
        ot{some(ddt), wide, es, "ddt"}, oa{da, (size_t)d * n * 4, 4, "da"}, ob{some(db), narrow, es, "db"}, oc{some(dc), narrow, es, "dc"},
        os{dskip, (size_t)d * 4, 4, "dskip"}, oz{z ? some(dz) : nullptr, wide, es, "dz"}, oi{ddt_bias, (size_t)d * 4, 4, "ddt_bias"},
        oh{dh0, state, 4, "dh0"}, ws{workspace, need, 16, "workspace"};
    st = rows > 0 ? check_args({au, at, aa, ab, ac, av, ay, ou, ot, oa, ob, oc, ws}, {as, az, ai, ar, al, ah, os, oz, oi, oh})
                  : check_args({aa, oa, ws}, {as, ai, al, ah, os, oi, oh});
    if (st == SCAN_OK) st = check_workspace("ssm_scan_bwd", workspace_bytes, need);
    if (st == SCAN_OK) st = check_alias({au, at, aa, ab, ac, as, az, ai, ar, al, av, ay, ah}, {ou, ot, oa, ob, oc, os, oz, oi, oh, ws});
    if (st != SCAN_OK) return st;
    ssm_layout(true, batch, length, d, n, groups, workspace, &k);
    k.batch = (int)batch, k.length = (int)length, k.d = d, k.n = n, k.groups = groups, k.per = d / groups, k.softplus = softplus != 0;
    k.u = u, k.dt = dt, k.b = b, k.c = c, k.z = z;
    k.u_stride = u_stride, k.dt_stride = dt_stride, k.b_stride = b_stride, k.c_stride = c_stride, k.z_stride = z_stride;
    k.a = a, k.skip = skip, k.dt_bias = dt_bias, k.reset = reset, k.lengths = lengths;
    k.saved = static_cast<float*>(const_cast<void*>(saved));
    k.dy = dy, k.dy_stride = dy_stride, k.dh = dh_final;
    k.du = du, k.ddt = ddt, k.db = db, k.dc = dc, k.dz = dz;
    k.da = da, k.dskip = dskip, k.ddt_bias = ddt_bias, k.dh0 = dh0;
    return device_status(launch_ssm_bwd(k, dtype == SCAN_F32, (hipStream_t)stream), "selective scan backward");
}

scan_status ssm_scan_step(int64_t batch, int d, int n, int groups, int dtype, int softplus, float* h, const void* u, int64_t u_stride,
                          const void* dt, int64_t dt_stride, const float* a, const void* b, int64_t b_stride, const void* c, int64_t c_stride,
                          const float* skip, const void* z, int64_t z_stride, const float* dt_bias, void* y, void* stream) {
    scan_status st = ssm_check("ssm_scan_step", batch, 1, d, n, groups, dtype, {u_stride, dt_stride, b_stride, c_stride, z_stride}, kMaxStride);
    if (st != SCAN_OK) return st;
    if (batch == 0) return SCAN_OK;
    const size_t es = dtype_size(dtype);
    const Arg oh{h, (size_t)batch * d * n * 4, 4, "h"}, au{u, span(batch, u_stride, d, es), es, "u"}, at{dt, span(batch, dt_stride, d, es), es, "dt"},
        aa{a, (size_t)d * n * 4, 4, "a"}, ab{b, span(batch, b_stride, groups * n, es), es, "b"}, ac{c, span(batch, c_stride, groups * n, es), es, "c"},
        as{skip, (size_t)d * 4, 4, "skip"}, az{z, span(batch, z_stride, d, es), es, "z"}, ai{dt_bias, (size_t)d * 4, 4, "dt_bias"},
        oy{y, (size_t)batch * d * es, es, "y"};
    st = check_args({oh, au, at, aa, ab, ac, oy}, {as, az, ai});
    if (st == SCAN_OK) st = check_alias({au, at, aa, ab, ac, as, az, ai}, {oh, oy});
    if (st != SCAN_OK) return st;
    SsmArgs k{};
    k.plan.ng = n <= SSM_STATES ? 1 : ssm_state_groups(n);  // lanes of a channel
    k.batch = (int)batch, k.length = 1, k.d = d, k.n = n, k.groups = groups, k.per = d / groups, k.softplus = softplus != 0;
    k.u = u, k.dt = dt, k.b = b, k.c = c, k.z = z;
    k.u_stride = u_stride, k.dt_stride = dt_stride, k.b_stride = b_stride, k.c_stride = c_stride, k.z_stride = z_stride;
    k.a = a, k.skip = skip, k.dt_bias = dt_bias;
    k.y = y, k.h = h;
    return device_status(launch_ssm_step(k, dtype == SCAN_F32, (hipStream_t)stream), "selective scan step");
}

// -------------------------------------------------- causal convolution ---
scan_status ssm_conv_fwd(int64_t batch, int64_t length, int d, int width, int dtype, int act, const void* x, int64_t x_stride, const float* w,
                         const float* bias, const void* state, const uint8_t* reset, const int32_t* lengths, void* y, void* state_out,
                         void* stream) {
    scan_status st = conv_check("ssm_conv_fwd", batch, length, d, width, dtype, act, {x_stride});
    if (st != SCAN_OK) return st;
    if (batch == 0) return SCAN_OK;
    const size_t es = dtype_size(dtype), sb = (size_t)batch * (width - 1) * d * es;
    const int64_t rows = batch * length;
    const auto some = [&](const void* p) { return rows > 0 ? p : nullptr; };
    const Arg ax{some(x), span(rows, x_stride, d, es), es, "x"}, aw{w, (size_t)d * width * 4, 4, "w"}, ab{bias, (size_t)d * 4, 4, "bias"},
        as{state, sb, es, "state"}, ar{some(reset), (size_t)rows, 1, "reset"}, al{lengths, (size_t)batch * 4, 4, "lengths"},
        oy{some(y), (size_t)rows * d * es, es, "y"}, os{state_out, sb, es, "state_out"};
    st = rows > 0 ? check_args({ax, aw, oy}, {ab, as, ar, al, os}) : check_args({aw}, {ab, as, al, os});
    if (st == SCAN_OK) st = check_alias({ax, aw, ab, as, ar, al}, {oy, os});
    if (st != SCAN_OK) return st;
    ConvArgs k{};
    conv_plan(batch, length, d, false, &k);
    k.batch = (int)batch, k.length = (int)length, k.d = d, k.width = width, k.act = act;
    k.x = x, k.x_stride = x_stride, k.w = w, k.bias = bias, k.state = state, k.reset = reset, k.lengths = lengths;
    k.y = y, k.state_out = state_out;
    return device_status(launch_conv_fwd(k, dtype == SCAN_F32, (hipStream_t)stream), "causal convolution");
}

size_t ssm_conv_bwd_workspace_bytes(int64_t batch, int64_t length, int d, int width) {
    return conv_fits(batch, length, d, width) ? conv_part_bytes(batch, length, d, width) : 0;
}

scan_status ssm_conv_bwd(int64_t batch, int64_t length, int d, int width, int dtype, int act, const void* x, int64_t x_stride, const float* w,
                         const float* bias, const void* state, const uint8_t* reset, const int32_t* lengths, const void* dy, int64_t dy_stride,
                         const void* dstate_out, void* dx, float* dw, float* dbias, void* dstate, void* workspace, size_t workspace_bytes,
                         void* stream) {
    scan_status st = conv_check("ssm_conv_bwd", batch, length, d, width, dtype, act, {x_stride, dy_stride});
    if (st != SCAN_OK) return st;
    const size_t es = dtype_size(dtype), sb = (size_t)batch * (width - 1) * d * es, need = conv_part_bytes(batch, length, d, width);
    const int64_t rows = batch * length;
    const auto some = [&](const void* p) { return rows > 0 ? p : nullptr; };
    const Arg ax{some(x), span(rows, x_stride, d, es), es, "x"}, aw{w, (size_t)d * width * 4, 4, "w"}, ab{bias, (size_t)d * 4, 4, "bias"},
        as{state, sb, es, "state"}, ar{some(reset), (size_t)rows, 1, "reset"}, al{lengths, (size_t)batch * 4, 4, "lengths"},
        ay{some(dy), span(rows, dy_stride, d, es), es, "dy"}, ao{dstate_out, sb, es, "dstate_out"}, ox{some(dx), (size_t)rows * d * es, es, "dx"},
        ow{dw, (size_t)d * width * 4, 4, "dw"}, ob{dbias, (size_t)d * 4, 4, "dbias"}, os{dstate, sb, es, "dstate"},
        ws{workspace, need, 16, "workspace"};
    st = rows > 0 ? check_args({ax, aw, ay, ox, ow, ws}, {ab, as, ar, al, ao, ob, os}) : check_args({aw, ow, ws}, {ab, as, al, ao, ob, os});
    if (st == SCAN_OK) st = check_workspace("ssm_conv_bwd", workspace_bytes, need);
    if (st == SCAN_OK) st = check_alias({ax, aw, ab, as, ar, al, ay, ao}, {ox, ow, ob, os, ws});
    if (st != SCAN_OK) return st;
    ConvArgs k{};
    conv_plan(batch, length, d, true, &k);
    k.batch = (int)batch, k.length = (int)length, k.d = d, k.width = width, k.act = act;
    k.x = x, k.x_stride = x_stride, k.w = w, k.bias = bias, k.state = state, k.reset = reset, k.lengths = lengths;
    k.dy = dy, k.dy_stride = dy_stride, k.dstate_out = dstate_out;
    k.dx = dx, k.dw = dw, k.dbias = dbias, k.dstate = dstate, k.part = static_cast<float*>(workspace);
    return device_status(launch_conv_bwd(k, dtype == SCAN_F32, (hipStream_t)stream), "causal convolution backward");
}

scan_status ssm_conv_step(int64_t batch, int d, int width, int dtype, int act, const void* x, int64_t x_stride, const float* w,
                          const float* bias, void* state, void* y, void* stream) {
    scan_status st = conv_check("ssm_conv_step", batch, 1, d, width, dtype, act, {x_stride});
    if (st != SCAN_OK) return st;
    if (batch == 0) return SCAN_OK;
    const size_t es = dtype_size(dtype);
    const Arg ax{x, span(batch, x_stride, d, es), es, "x"}, aw{w, (size_t)d * width * 4, 4, "w"}, ab{bias, (size_t)d * 4, 4, "bias"},
        os{state, (size_t)batch * (width - 1) * d * es, es, "state"}, oy{y, (size_t)batch * d * es, es, "y"};
    st = check_args({ax, aw, os, oy}, {ab});
    if (st == SCAN_OK) st = check_alias({ax, aw, ab}, {os, oy});
    if (st != SCAN_OK) return st;
    ConvArgs k{};
    k.batch = (int)batch, k.length = 1, k.d = d, k.width = width, k.act = act, k.tokens = 1, k.pieces = 1;
    k.x = x, k.x_stride = x_stride, k.w = w, k.bias = bias, k.state = state, k.y = y;
    return device_status(launch_conv_step(k, dtype == SCAN_F32, (hipStream_t)stream), "causal convolution step");
}

}  // extern "C"
