// lm_capi.cpp -- the C ABI of the language-model operators (lm_ops.h):
// argument validation, workspace layout and kernel sequencing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <vector>

#include "capi_check.hpp"
#include "lm.hpp"
#include "lm_ce_plan.hpp"
#include "lm_ops.h"

namespace lrs {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 40;
// a tile's 256 rows, or 64 steps, stay inside the 31-bit offsets of a buffer descriptor
constexpr int64_t kMaxCeStride = (int64_t)1 << 21;

scan_status norm_shape(const char* fn, int64_t rows, int d, int st, int br, int act, const void* gate,
                       const float* w_post, const float* scale, std::initializer_list<int64_t> strides) {
    if (rows < 0 || rows > kMaxRows || d < 1 || d > LM_NORM_MAX_D)
        return fail(SCAN_ERR_SHAPE, std::string(fn) + ": unsupported shape rows=" + std::to_string(rows) + " d=" +
                                        std::to_string(d) + " (need 1 <= d <= " + std::to_string(LM_NORM_MAX_D) + ")");
    if (!dtype_ok(st) || !dtype_ok(br))
        return fail(SCAN_ERR_SHAPE, std::string(fn) + ": dtypes must be SCAN_BF16 or SCAN_F32");
    if (act < LM_GATE_NONE || act > LM_GATE_SILU)
        return fail(SCAN_ERR_SHAPE, std::string(fn) + ": gate_act must be LM_GATE_NONE, _SIGMOID or _SILU");
    if (rows > 0 && (act == LM_GATE_NONE) != (gate == nullptr))
        return fail(gate ? SCAN_ERR_SHAPE : SCAN_ERR_NULL,
                    std::string(fn) + ": a gate is given with, and only with, a gate activation");
    if ((w_post == nullptr) != (scale == nullptr))
        return fail(SCAN_ERR_NULL, std::string(fn) + ": w_post and scale are given together or not at all");
    for (int64_t s : strides)
        if (s < 0 || s > kMaxRows) return fail(SCAN_ERR_SHAPE, std::string(fn) + ": row strides must not be negative");
    return SCAN_OK;
}

size_t norm_part_bytes(int64_t rows, int d) {
    return std::max<size_t>(256, (size_t)(rows > 0 ? lm_norm_bwd_blocks(rows, d) : 0) * 2 * d * sizeof(float));
}

// Buffers of the linear cross entropy inside the caller's workspace (base NULL: sizes only).
size_t ce_layout(bool bwd, int n, int d, int v, void* base, CeArgs* a) {
    char* p = static_cast<char*>(base);
    size_t off = 0;
    const auto take = [&](size_t bytes) {
        void* at = p ? p + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    if (bwd) {
        const CePlan pl = ce_plan(n, d, v);
        a->scale = static_cast<float*>(take(4));
        a->active = static_cast<int*>(take(4));
        a->list = static_cast<int*>(take((size_t)n * 4));
        a->place = static_cast<int*>(take((size_t)n * 4));
        a->token = static_cast<CeToken*>(take((size_t)n * sizeof(CeToken)));
        a->packed = take((size_t)n * d * 2);
        a->dz = take((size_t)(pl.few ? pl.few : n) * pl.chunk * 2);
        a->dh_part = static_cast<float*>(take((size_t)pl.splits * n * d * 4));
    } else {
        a->part = static_cast<float*>(take((size_t)ce_parts(n, d, v) * n * 8));
        a->picked = static_cast<float*>(take((size_t)n * 4));
    }
    return std::max<size_t>(off, 256);
}

scan_status ce_check(const char* fn, int64_t n, int d, int64_t v, double cap, int64_t h_stride) {
    if (!ce_shape(n, d, v))
        return fail(SCAN_ERR_SHAPE, std::string(fn) + ": unsupported shape n=" + std::to_string(n) + " d=" + std::to_string(d) +
                                        " v=" + std::to_string(v) + " (need v >= 1, 8 <= d <= 65536 a multiple of 8, n <= 2^26 - 16, n d <= 2^34 - 1024)");
    if (!(cap >= 0.0) || !std::isfinite((float)cap) || (cap > 0.0 && (float)cap < 1e-30f))
        return fail(SCAN_ERR_SHAPE, std::string(fn) + ": softcap must be 0 (none) or a positive number");
    if (n > 0 && (h_stride % 8 != 0 || h_stride < 0 || h_stride > kMaxCeStride))
        return fail(SCAN_ERR_SHAPE, std::string(fn) + ": the rows of h must lie a multiple of 8 elements apart");
    return SCAN_OK;
}

static_assert(LM_EMBED_MAX_V == EMBED_MOST_V, "the header's limit");
// Launches of 64 threads for a token, or two for a row of the vocabulary in whole workgroups, along x, and a workgroup for 256 columns along y.
bool embed_shape(int64_t n, int d, int64_t v) {
    return n >= 0 && d >= 1 && v >= 1 && n <= (1 << 26) - 64 && v <= EMBED_MOST_V && d <= (1 << 23);
}
scan_status embed_refuse(const char* fn, int64_t n, int d, int64_t v) {
    return fail(SCAN_ERR_SHAPE, std::string(fn) + ": unsupported shape n=" + std::to_string(n) + " d=" + std::to_string(d) + " v=" +
                                    std::to_string(v) + " (need 1 <= d <= 2^23, 1 <= v <= " + std::to_string(EMBED_MOST_V) + ", n <= 2^26 - 64)");
}

// The gradient's buffers inside the caller's workspace (base NULL: sizes only).
size_t embed_layout(int64_t n, int d, int64_t v, void* base, EmbedArgs* a) {
    char* p = static_cast<char*>(base);
    size_t off = 0;
    const auto take = [&](size_t bytes) {
        void* at = p ? p + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    a->start = static_cast<int*>(take((size_t)(v + 1) * 4));
    a->order = static_cast<int*>(take((size_t)n * 4));
    a->part = static_cast<float*>(take((size_t)ceil_div(n, EMBED_RUN) * 2 * d * 4));
    return std::max<size_t>(off, 256);
}

}  // namespace
}  // namespace lrs

using namespace lrs;

extern "C" {

// -------------------------------------------------------- block norms ---
scan_status lm_block_norm_fwd(int64_t rows, int d, int stream_dtype, int branch_dtype, int gate_act, double eps,
                              const void* x, int64_t x_stride, const void* y, int64_t y_stride, const void* gate,
                              int64_t gate_stride, const float* w_post, const float* scale, const float* w_pre,
                              void* r, void* n, float* stats, void* stream) {
    scan_status st = norm_shape("lm_block_norm_fwd", rows, d, stream_dtype, branch_dtype, gate_act, gate, w_post,
                                scale, {x_stride, y_stride, gate_stride});
    if (st != SCAN_OK) return st;
    if (!(eps >= 0.0)) return fail(SCAN_ERR_SHAPE, "lm_block_norm_fwd: eps must not be negative");
    if (rows == 0) return SCAN_OK;
    const size_t ss = dtype_size(stream_dtype), bs = dtype_size(branch_dtype), rd = (size_t)rows * d, dw = (size_t)d * 4;
    const Arg ax{x, span(rows, x_stride, d, ss), ss, "x"}, ay{y, span(rows, y_stride, d, bs), bs, "y"},
        ag{gate, span(rows, gate_stride, d, bs), bs, "gate"}, a1{w_post, dw, 4, "w_post"}, as{scale, dw, 4, "scale"},
        a2{w_pre, dw, 4, "w_pre"}, ar{r, rd * ss, ss, "r"}, an{n, rd * bs, bs, "n"},
        at{stats, (size_t)rows * 8, 4, "stats"};
    st = check_args({ax, ay, a2, ar, an, at}, {ag, a1, as});
    if (st != SCAN_OK) return st;
    // r may be x itself: all of a row is read before any of it is written.  Not by each lane its own elements (where d is no
    // multiple of 4 the lane at the row's end reads its neighbour's too), but because r's norm, which needs them all, stands between:
    // with a barrier where a row is several waves', and a wave's lanes run together.
    const bool in_place = r == x && (x_stride == d || rows == 1);
    st = check_alias({in_place ? Arg{nullptr, 0, 1, "x"} : ax, ay, ag, a1, as, a2}, {ar, an, at});
    if (st != SCAN_OK) return st;
    NormArgs a{};
    a.rows = rows;
    a.d = d;
    a.gate_act = gate_act;
    a.eps = (float)eps;
    a.x = x, a.y = y, a.gate = gate;
    a.x_stride = x_stride, a.y_stride = y_stride, a.gate_stride = gate_stride;
    a.w_post = w_post, a.scale = scale, a.w_pre = w_pre;
    a.r = r, a.n = n, a.stats = stats;
    return device_status(launch_norm_fwd(a, stream_dtype == SCAN_F32, branch_dtype == SCAN_F32, (hipStream_t)stream),
                         "block norm");
}

size_t lm_block_norm_bwd_workspace_bytes(int64_t rows, int d) {
    if (rows < 0 || rows > kMaxRows || d < 1 || d > LM_NORM_MAX_D) return 0;
    return norm_part_bytes(rows, d);
}

scan_status lm_block_norm_bwd(int64_t rows, int d, int stream_dtype, int branch_dtype, int gate_act, const void* x,
                              int64_t x_stride, const void* y, int64_t y_stride, const void* gate,
                              int64_t gate_stride, const float* w_post, const float* scale, const float* w_pre,
                              const float* stats, const void* dr, int64_t dr_stride, const void* dn,
                              int64_t dn_stride, void* dx, void* dy, void* dgate, float* dw_post, float* dscale,
                              float* dw_pre, void* workspace, size_t workspace_bytes, void* stream) {
    scan_status st = norm_shape("lm_block_norm_bwd", rows, d, stream_dtype, branch_dtype, gate_act, gate, w_post,
                                scale, {x_stride, y_stride, gate_stride, dr_stride, dn_stride});
    if (st != SCAN_OK) return st;
    if (gate && !dgate && rows > 0) return fail(SCAN_ERR_NULL, "dgate is NULL");
    if (w_post && (!dw_post || !dscale)) return fail(SCAN_ERR_NULL, "dw_post or dscale is NULL");
    const size_t ss = dtype_size(stream_dtype), bs = dtype_size(branch_dtype), rd = (size_t)rows * d, dw = (size_t)d * 4;
    const size_t need = norm_part_bytes(rows, d);
    const Arg ax{x, span(rows, x_stride, d, ss), ss, "x"}, ay{y, span(rows, y_stride, d, bs), bs, "y"},
        ag{gate, span(rows, gate_stride, d, bs), bs, "gate"}, a1{w_post, dw, 4, "w_post"}, as{scale, dw, 4, "scale"},
        a2{w_pre, dw, 4, "w_pre"}, at{stats, (size_t)rows * 8, 4, "stats"},
        ar{dr, span(rows, dr_stride, d, ss), ss, "dr"}, an{dn, span(rows, dn_stride, d, bs), bs, "dn"},
        ox{dx, rd * ss, ss, "dx"}, oy{dy, rd * bs, bs, "dy"}, og{gate ? dgate : nullptr, rd * bs, bs, "dgate"},
        o1{w_post ? dw_post : nullptr, dw, 4, "dw_post"}, os{w_post ? dscale : nullptr, dw, 4, "dscale"},
        o2{dw_pre, dw, 4, "dw_pre"}, ws{workspace, need, 16, "workspace"};
    if (rows > 0) {
        st = check_args({ax, ay, a2, at, ox, oy, o2, ws}, {ag, a1, as, ar, an, og, o1, os});
    } else {
        st = check_args({a2, o2, ws}, {a1, as, o1, os});
    }
    if (st != SCAN_OK) return st;
    if (workspace_bytes < need)
        return fail(SCAN_ERR_WORKSPACE, "lm_block_norm_bwd: workspace_bytes " + std::to_string(workspace_bytes) +
                                            " < " + std::to_string(need));
    st = check_alias({ax, ay, ag, a1, as, a2, at, ar, an}, {ox, oy, og, o1, os, o2, ws});
    if (st != SCAN_OK) return st;
    NormArgs a{};
    a.rows = rows;
    a.d = d;
    a.gate_act = gate_act;
    a.x = x, a.y = y, a.gate = gate;
    a.x_stride = x_stride, a.y_stride = y_stride, a.gate_stride = gate_stride;
    a.w_post = w_post, a.scale = scale, a.w_pre = w_pre;
    a.stats = const_cast<float*>(stats);
    a.dr = dr, a.dn = dn;
    a.dr_stride = dr_stride, a.dn_stride = dn_stride;
    a.dx = dx, a.dy = dy, a.dgate = dgate;
    a.part = static_cast<float*>(workspace);
    return device_status(launch_norm_bwd(a, stream_dtype == SCAN_F32, branch_dtype == SCAN_F32, dw_post, dscale,
                                         dw_pre, (hipStream_t)stream),
                         "block norm backward");
}

// ----------------------------------------------- linear cross entropy ---
size_t lm_linear_ce_workspace_bytes(int64_t n, int d, int64_t v, int backward) {
    if (!ce_shape(n, d, v)) return 0;
    CeArgs a{};
    return ce_layout(backward != 0, (int)n, d, (int)v, nullptr, &a);
}

scan_status lm_linear_ce_fwd(int64_t n, int d, int64_t v, double softcap, const void* h, int64_t h_stride, const void* w,
                             const int64_t* target, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
    scan_status st = ce_check("lm_linear_ce_fwd", n, d, v, softcap, h_stride);
    if (st != SCAN_OK) return st;
    if (n == 0) return SCAN_OK;
    CeArgs a{};
    const size_t need = ce_layout(false, (int)n, d, (int)v, nullptr, &a), nb = (size_t)n * 4;
    const Arg ah{h, span(n, h_stride, d, 2), 16, "h"}, aw{w, (size_t)v * d * 2, 16, "w"}, at{target, (size_t)n * 8, 8, "target"},
        ol{loss, nb, 4, "loss"}, oe{lse, nb, 4, "lse"}, ws{workspace, need, 16, "workspace"};
    st = check_args({ah, aw, at, ol, oe, ws}, {});
    if (st != SCAN_OK) return st;
    if (workspace_bytes < need)
        return fail(SCAN_ERR_WORKSPACE, "lm_linear_ce_fwd: workspace_bytes " + std::to_string(workspace_bytes) + " < " +
                                            std::to_string(need));
    st = check_alias({ah, aw, at}, {ol, oe, ws});
    if (st != SCAN_OK) return st;
    ce_layout(false, (int)n, d, (int)v, workspace, &a);
    a.n = (int)n, a.d = d, a.v = (int)v, a.cap = (float)softcap;
    a.h = h, a.h_stride = h_stride, a.w = w, a.target = target;
    a.loss = loss, a.lse = lse;
    return device_status(launch_ce_fwd(a, (hipStream_t)stream), "linear cross entropy");
}

scan_status lm_linear_ce_bwd(int64_t n, int d, int64_t v, double softcap, const void* h, int64_t h_stride, const void* w,
                             const int64_t* target, const float* lse, const float* dloss, const float* dlse, void* dh,
                             void* dw, int grad_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    scan_status st = ce_check("lm_linear_ce_bwd", n, d, v, softcap, h_stride);
    if (st != SCAN_OK) return st;
    if (!dtype_ok(grad_dtype)) return fail(SCAN_ERR_SHAPE, "lm_linear_ce_bwd: grad_dtype must be SCAN_BF16 or SCAN_F32");
    CeArgs a{};
    const size_t need = ce_layout(true, (int)n, d, (int)v, nullptr, &a), nb = (size_t)n * 4, g = dtype_size(grad_dtype);
    const Arg ah{h, span(n, h_stride, d, 2), 16, "h"}, aw{w, (size_t)v * d * 2, 16, "w"}, at{target, (size_t)n * 8, 8, "target"},
        ae{lse, nb, 4, "lse"}, al{dloss, nb, 4, "dloss"}, az{dlse, nb, 4, "dlse"}, oh{dh, (size_t)n * d * g, 16, "dh"},
        ow{dw, (size_t)v * d * g, 16, "dw"}, ws{workspace, need, 16, "workspace"};
    st = n > 0 ? check_args({ah, aw, at, ae, al, oh, ow, ws}, {az}) : check_args({ow}, {});
    if (st != SCAN_OK) return st;
    if (workspace_bytes < need && n > 0)
        return fail(SCAN_ERR_WORKSPACE, "lm_linear_ce_bwd: workspace_bytes " + std::to_string(workspace_bytes) + " < " +
                                            std::to_string(need));
    st = check_alias({ah, aw, at, ae, al, az}, {oh, ow, ws});
    if (st != SCAN_OK) return st;
    ce_layout(true, (int)n, d, (int)v, workspace, &a);
    a.n = (int)n, a.d = d, a.v = (int)v, a.cap = (float)softcap;
    a.h = h, a.h_stride = h_stride, a.w = w, a.target = target;
    a.lse_in = lse, a.dloss = dloss, a.dlse = dlse;
    a.dh = dh, a.dw = dw, a.grad_f32 = grad_dtype == SCAN_F32;
    return device_status(launch_ce_bwd(a, (hipStream_t)stream), "linear cross entropy backward");
}

// --------------------------------------------------------------- AdamW ---
scan_status lm_adamw_step(int count, int param_dtype, int grad_dtype, int state_bits, void* const* p,
                          const void* const* g, void* const* m, void* const* v, float* const* master,
                          float* const* m_scale, float* const* v_scale, const int64_t* n, const double* decay,
                          double lr, double beta1, double beta2, double eps, int64_t step, void* stream) {
    if (count < 0) return fail(SCAN_ERR_SHAPE, "lm_adamw_step: count must not be negative");
    if (!dtype_ok(param_dtype) || !dtype_ok(grad_dtype))
        return fail(SCAN_ERR_SHAPE, "lm_adamw_step: dtypes must be SCAN_BF16 or SCAN_F32");
    if (state_bits != 8 && state_bits != 32) return fail(SCAN_ERR_SHAPE, "lm_adamw_step: state_bits must be 8 or 32");
    if (step < 1) return fail(SCAN_ERR_SHAPE, "lm_adamw_step: step counts from 1");
    if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(lr))
        return fail(SCAN_ERR_SHAPE, "lm_adamw_step: need 0 <= beta < 1, eps >= 0 and a finite lr");
    if (count == 0) return SCAN_OK;
    const bool bits8 = state_bits == 8;
    if (!p || !g || !m || !v || !n || !decay || (bits8 && (!m_scale || !v_scale)))
        return fail(SCAN_ERR_NULL, "lm_adamw_step: a list is NULL");
    const size_t ps = dtype_size(param_dtype), gs = dtype_size(grad_dtype), ms = bits8 ? 1 : 4;
    struct Extent {
        uintptr_t a, b;
        int i;
        const char* name;
        bool out;
    };
    std::vector<Extent> ext;
    ext.reserve((size_t)count * 7);
    for (int i = 0; i < count; ++i) {
        const auto at = [i] { return " of tensor " + std::to_string(i); };
        if (n[i] < 0 || n[i] > kMaxRows) return fail(SCAN_ERR_SHAPE, "lm_adamw_step: unsupported size" + at());
        if (n[i] == 0) continue;
        const size_t k = (size_t)n[i], kb = (size_t)ceil_div(n[i], LM_ADAMW_BLOCK) * 4;
        const Arg args[7] = {{p[i], k * ps, ps, "p"},
                             {g[i], k * gs, gs, "g"},
                             {m[i], k * ms, ms, "m"},
                             {v[i], k * ms, ms, "v"},
                             {master ? master[i] : nullptr, k * 4, 4, "master"},
                             {bits8 ? m_scale[i] : nullptr, kb, 4, "m_scale"},
                             {bits8 ? v_scale[i] : nullptr, kb, 4, "v_scale"}};
        for (int j = 0; j < 7; ++j) {
            const bool wanted = j < 4 || (j == 4 ? master != nullptr : bits8);
            if (!wanted) continue;
            const Arg& a = args[j];
            if (!a.p) return fail(SCAN_ERR_NULL, std::string(a.name) + at() + " is NULL");
            if ((uintptr_t)a.p & (a.align - 1))
                return fail(SCAN_ERR_ALIGN, std::string(a.name) + at() + " is not " + std::to_string(a.align) +
                                                "-byte aligned");
            ext.push_back({(uintptr_t)a.p, (uintptr_t)a.p + a.n, i, a.name, j != 1});
        }
    }
    // every extent but a gradient is written: after sorting by address, an
    // overlap shows between an extent and the furthest end before it
    std::sort(ext.begin(), ext.end(), [](const Extent& x, const Extent& y) { return x.a < y.a; });
    const Extent *end_any = nullptr, *end_out = nullptr;  // furthest ends so far, of all and of the written ones
    for (const Extent& e : ext) {
        const Extent* hit = e.out ? end_any : end_out;
        if (hit && e.a < hit->b)
            return fail(SCAN_ERR_ALIAS, std::string(e.name) + " of tensor " + std::to_string(e.i) + " overlaps " +
                                            hit->name + " of tensor " + std::to_string(hit->i));
        if (!end_any || e.b > end_any->b) end_any = &e;
        if (e.out && (!end_out || e.b > end_out->b)) end_out = &e;
    }
    AdamwArgs a;
    a.b1 = (float)beta1, a.c1 = (float)(1.0 - beta1), a.b2 = (float)beta2, a.c2 = (float)(1.0 - beta2);
    a.step_size = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
    a.root_scale = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
    a.eps = (float)eps;
    a.count = 0;
    uint64_t blocks = 0;
    // a launch holds ADAMW_LAUNCH tensors and workgroups of 256 threads; a
    // tensor that does not fit what is left of them is cut at a whole chunk
    constexpr uint64_t kMost = MOST_THREADS / 256;
    auto flush = [&]() -> hipError_t {
        if (a.count == 0) return hipSuccess;
        const hipError_t e = launch_adamw(a, (uint32_t)blocks, param_dtype == SCAN_F32, grad_dtype == SCAN_F32,
                                          master != nullptr, bits8, (hipStream_t)stream);
        a.count = 0;
        blocks = 0;
        return e;
    };
    for (int i = 0; i < count; ++i) {
        int64_t done = 0;
        while (done < n[i]) {
            if (a.count == ADAMW_LAUNCH || blocks == kMost) {
                scan_status st = device_status(flush(), "adamw");
                if (st != SCAN_OK) return st;
            }
            const int64_t left = n[i] - done;
            const uint64_t want = (uint64_t)ceil_div(left, ADAMW_CHUNK), take = std::min(want, kMost - blocks);
            const int64_t k = std::min<int64_t>(left, (int64_t)take * ADAMW_CHUNK);
            const int c = a.count++;
            a.start[c] = (uint32_t)blocks;
            a.decay[c] = (float)(lr * decay[i]);
            a.n[c] = k;
            a.p[c] = (char*)p[i] + done * ps;
            a.g[c] = (const char*)g[i] + done * gs;
            a.m[c] = (char*)m[i] + done * ms;
            a.v[c] = (char*)v[i] + done * ms;
            a.master[c] = master ? master[i] + done : nullptr;
            a.m_scale[c] = bits8 ? m_scale[i] + done / LM_ADAMW_BLOCK : nullptr;
            a.v_scale[c] = bits8 ? v_scale[i] + done / LM_ADAMW_BLOCK : nullptr;
            blocks += take;
            done += k;
        }
    }
    return device_status(flush(), "adamw");
}

// --------------------------------------------------- embedding lookup ---
size_t lm_embed_bwd_workspace_bytes(int64_t n, int d, int64_t v) {
    if (!embed_shape(n, d, v)) return 0;
    EmbedArgs a{};
    return embed_layout(n, d, v, nullptr, &a);
}

scan_status lm_embed_fwd(int64_t n, int d, int64_t v, int w_dtype, int out_dtype, double scale, const int64_t* tokens, const void* w,
                         void* out, void* stream) {
    if (!embed_shape(n, d, v)) return embed_refuse("lm_embed_fwd", n, d, v);
    if (!dtype_ok(w_dtype) || !dtype_ok(out_dtype)) return fail(SCAN_ERR_SHAPE, "lm_embed_fwd: dtypes must be SCAN_BF16 or SCAN_F32");
    if (!std::isfinite((float)scale)) return fail(SCAN_ERR_SHAPE, "lm_embed_fwd: scale must be finite");
    if (n == 0) return SCAN_OK;
    const size_t ws = dtype_size(w_dtype), os = dtype_size(out_dtype);
    const Arg at{tokens, (size_t)n * 8, 8, "tokens"}, aw{w, (size_t)v * d * ws, ws, "w"}, ao{out, (size_t)n * d * os, os, "out"};
    scan_status st = check_args({at, aw, ao}, {});
    if (st == SCAN_OK) st = check_alias({at, aw}, {ao});
    if (st != SCAN_OK) return st;
    EmbedArgs a{};
    a.n = n, a.v = v, a.d = d, a.scale = (float)scale;
    a.tokens = tokens, a.w = w, a.out = out;
    return device_status(launch_embed_fwd(a, w_dtype == SCAN_F32, out_dtype == SCAN_F32, (hipStream_t)stream), "embedding");
}

scan_status lm_embed_bwd(int64_t n, int d, int64_t v, int out_dtype, int grad_dtype, double scale, const int64_t* tokens,
                         const void* dout, int64_t dout_stride, int accumulate, void* dw, void* workspace, size_t workspace_bytes,
                         void* stream) {
    if (!embed_shape(n, d, v)) return embed_refuse("lm_embed_bwd", n, d, v);
    if (!dtype_ok(out_dtype) || !dtype_ok(grad_dtype)) return fail(SCAN_ERR_SHAPE, "lm_embed_bwd: dtypes must be SCAN_BF16 or SCAN_F32");
    if (!std::isfinite((float)scale)) return fail(SCAN_ERR_SHAPE, "lm_embed_bwd: scale must be finite");
    if (n > 0 && (dout_stride < 0 || dout_stride > kMaxRows)) return fail(SCAN_ERR_SHAPE, "lm_embed_bwd: row strides must not be negative");
    const size_t os = dtype_size(out_dtype), gs = dtype_size(grad_dtype);
    EmbedArgs a{};
    const size_t need = embed_layout(n, d, v, nullptr, &a);
    const Arg at{tokens, (size_t)n * 8, 8, "tokens"}, ao{dout, span(n, dout_stride, d, os), os, "dout"}, aw{dw, (size_t)v * d * gs, gs, "dw"},
        ws{workspace, need, 16, "workspace"};
    scan_status st = n > 0 ? check_args({at, ao, aw, ws}, {}) : check_args({aw}, {});
    if (st != SCAN_OK) return st;
    if (n > 0 && workspace_bytes < need)
        return fail(SCAN_ERR_WORKSPACE, "lm_embed_bwd: workspace_bytes " + std::to_string(workspace_bytes) + " < " + std::to_string(need));
    if (n > 0) st = check_alias({at, ao}, {aw, ws});
    if (st != SCAN_OK) return st;
    if (n == 0 && accumulate) return SCAN_OK;
    embed_layout(n, d, v, workspace, &a);
    a.n = n, a.v = v, a.d = d, a.scale = (float)scale, a.add = accumulate != 0;
    a.tokens = tokens, a.dout = dout, a.dout_stride = dout_stride, a.dw = dw;
    return device_status(launch_embed_bwd(a, out_dtype == SCAN_F32, grad_dtype == SCAN_F32, (hipStream_t)stream), "embedding backward");
}

}  // extern "C"
