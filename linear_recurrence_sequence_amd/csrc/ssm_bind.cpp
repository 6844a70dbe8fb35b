// ssm_bind.cpp -- the usual calls of ssm.py without its per-tensor Python work,
// as lm_bind.cpp makes those of lm.py: a decoding step's scan takes 4 us on the GPU, and
// looking at its ten tensors from Python took 20.
#include "lm_bind.hpp"

#include "ssm_ops.h"

namespace lrs_bind {
namespace {

// Row stride of b or c [..., groups, n], whose rows' values are dense.
int64_t group_stride(const Tensor& t) {
    const int64_t g = t.size(-2), n = t.size(-1);
    if (t.is_contiguous()) return g * n;
    need((n == 1 || t.stride(-1) == 1) && (g == 1 || t.stride(-2) == n));
    int64_t step = -1, reach = 0;
    for (int64_t i = t.dim() - 3; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (step < 0) step = t.stride(i);
        else need(t.stride(i) == reach);
        reach = t.stride(i) * t.size(i);
    }
    return step < 0 ? g * n : step;
}

struct Flags {
    const uint8_t* reset = nullptr;
    const int32_t* lengths = nullptr;
    Flags(PyObject* r, PyObject* l, int64_t batch, int64_t length, const c10::Device& dev) {
        if (r != Py_None) {
            const Tensor& t = tensor(r);
            need(t.dim() == 2 && t.size(0) == batch && t.size(1) == length && (t.scalar_type() == at::kByte || t.scalar_type() == at::kBool));
            reset = static_cast<const uint8_t*>(dense(t, t.scalar_type(), dev));
        }
        if (l != Py_None) {
            const Tensor& t = tensor(l);
            need(t.dim() == 1 && t.size(0) == batch);
            lengths = static_cast<const int32_t*>(dense(t, at::kInt, dev));
        }
    }
};

struct Scan {
    const Tensor &u, &A, &B, &C;
    c10::Device dev;
    int64_t batch = 0, length = 1, d = 0, n = 0, groups = 0, sb = 0, sc = 0;
    at::ScalarType type;
    int dtype;
    Matrix mu, mdt, mz;
    const float *pa, *skip, *bias;
    void *pb, *pc;
    // a: u, dt, a, b, c, d, z, dt_bias
    Scan(PyObject* const* a, int dims)
        : u(tensor(a[0])), A(tensor(a[2])), B(tensor(a[3])), C(tensor(a[4])), dev(u.device()), type(u.scalar_type()), dtype(code(type)) {
        need(dev.is_cuda() && u.dim() == dims && A.dim() == 2 && B.dim() == dims + 1 && C.sizes() == B.sizes());
        batch = u.size(0), d = u.size(-1), n = A.size(1), groups = B.size(-2);
        if (dims == 3) length = u.size(1);
        need(d >= 1 && d <= (1 << 21) && A.size(0) == d && n >= 1 && n <= SSM_MAX_STATE && B.size(-1) == n && B.size(0) == batch &&
             (dims == 2 || B.size(1) == length) && groups >= 1 && groups <= d);
        mu = {u.data_ptr(), row_stride(u)};
        mdt = matrix(a[1], u, type);
        mz = matrix(a[6], u, type);
        need(mdt.p || batch * length == 0);
        pa = static_cast<const float*>(dense(A, at::kFloat, dev));
        need(B.scalar_type() == type && C.scalar_type() == type && B.device() == dev && C.device() == dev);
        pb = B.data_ptr(), pc = C.data_ptr();
        sb = group_stride(B), sc = group_stride(C);
        skip = vec(a[5], d, dev);
        bias = vec(a[7], d, dev);
    }
    const float* state(PyObject* o) const {
        if (o == Py_None) return nullptr;
        const Tensor& t = tensor(o);
        need(t.dim() == 3 && t.size(0) == batch && t.size(1) == d && t.size(2) == n);
        return static_cast<const float*>(dense(t, at::kFloat, dev));
    }
    Tensor workspace(int backward) const {
        const size_t bytes = ssm_scan_workspace_bytes(batch, length, (int)d, (int)n, (int)groups, backward);
        need(bytes > 0);
        return empty({(int64_t)bytes}, at::kByte, dev);
    }
};

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    need(v >= 0);
    return v == 1;
}

struct Conv {
    const Tensor &x, &w;
    c10::Device dev;
    int64_t batch = 0, length = 1, d = 0, width = 0, stride = 0;
    at::ScalarType type;
    int dtype;
    const float *pw, *bias;
    // a: x, w, bias
    Conv(PyObject* const* a, int dims) : x(tensor(a[0])), w(tensor(a[1])), dev(x.device()), type(x.scalar_type()), dtype(code(type)) {
        need(dev.is_cuda() && x.dim() == dims && w.dim() == 2);
        batch = x.size(0), d = x.size(-1), width = w.size(1), stride = row_stride(x);
        if (dims == 3) length = x.size(1);
        need(d >= 1 && d <= (1 << 24) && w.size(0) == d && width >= 2 && width <= CONV_MAX_WIDTH);
        pw = static_cast<const float*>(dense(w, at::kFloat, dev));
        bias = vec(a[2], d, dev);
    }
    void* state(PyObject* o) const {
        if (o == Py_None) return nullptr;
        const Tensor& t = tensor(o);
        need(t.dim() == 3 && t.size(0) == batch && t.size(1) == width - 1 && t.size(2) == d);
        return dense(t, type, dev);
    }
};

}  // namespace

// (u, dt, a, b, c, d, z, dt_bias, h0, softplus, reset, lengths, want_saved, stream) -> (y, h_final, saved or None)
LRS_BOUND(ssm_scan_fwd) {
    return guarded([&]() -> PyObject* {
        need(count == 14);
        const Scan k(a, 3);
        const Flags f(a[10], a[11], k.batch, k.length, k.dev);
        const float* h0 = k.state(a[8]);
        Tensor y = empty(k.u.sizes(), k.type, k.dev), h = empty({k.batch, k.d, k.n}, at::kFloat, k.dev), ws = k.workspace(0), saved;
        if (truth(a[12])) {
            const size_t bytes = ssm_scan_saved_bytes(k.batch, k.length, (int)k.d, (int)k.n, (int)k.groups);
            need(bytes > 0);
            saved = empty({(int64_t)bytes}, at::kByte, k.dev);
        }
        const scan_status s = ::ssm_scan_fwd(k.batch, k.length, (int)k.d, (int)k.n, (int)k.groups, k.dtype, truth(a[9]), k.mu.p, k.mu.stride, k.mdt.p,
                                           k.mdt.stride, k.pa, k.pb, k.sb, k.pc, k.sc, k.skip, k.mz.p, k.mz.stride, k.bias, h0, f.reset, f.lengths,
                                           y.data_ptr(), static_cast<float*>(h.data_ptr()), saved.defined() ? saved.data_ptr() : nullptr,
                                           ws.data_ptr(), (size_t)ws.numel(), stream_of(a[13], k.dev));
        if (s != SCAN_OK) return status(s);
        PyObject* kept = Py_None;
        if (saved.defined()) kept = THPVariable_Wrap(saved);
        else Py_INCREF(Py_None);
        return Py_BuildValue("(NNN)", THPVariable_Wrap(y), THPVariable_Wrap(h), kept);
    });
}

// (u, dt, a, b, c, d, z, dt_bias, saved, dy, dh_final, softplus, reset, lengths, want_dh0, stream) -> dict
LRS_BOUND(ssm_scan_bwd) {
    return guarded([&]() -> PyObject* {
        need(count == 16);
        const Scan k(a, 3);
        const Flags f(a[12], a[13], k.batch, k.length, k.dev);
        const Tensor& saved = tensor(a[8]);
        need(saved.numel() == (int64_t)ssm_scan_saved_bytes(k.batch, k.length, (int)k.d, (int)k.n, (int)k.groups) && saved.dim() == 1);
        const void* ps = dense(saved, at::kByte, k.dev);
        need(a[9] != Py_None);
        const Matrix dy = matrix(a[9], k.u, k.type);
        const float* dh = k.state(a[10]);
        const auto wide = [&] { return empty(k.u.sizes(), k.type, k.dev); };
        const auto f32 = [](const Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; };
        Tensor du = wide(), ddt = wide(), dz, da = empty({k.d, k.n}, at::kFloat, k.dev), db = empty(k.B.sizes(), k.type, k.dev),
               dc = empty(k.B.sizes(), k.type, k.dev), dd, dbias, dh0, ws = k.workspace(1);
        if (a[6] != Py_None) dz = wide();
        if (k.skip) dd = empty({k.d}, at::kFloat, k.dev);
        if (k.bias) dbias = empty({k.d}, at::kFloat, k.dev);
        if (truth(a[14])) dh0 = empty({k.batch, k.d, k.n}, at::kFloat, k.dev);
        const scan_status s = ::ssm_scan_bwd(k.batch, k.length, (int)k.d, (int)k.n, (int)k.groups, k.dtype, truth(a[11]), k.mu.p, k.mu.stride, k.mdt.p,
                                           k.mdt.stride, k.pa, k.pb, k.sb, k.pc, k.sc, k.skip, k.mz.p, k.mz.stride, k.bias, f.reset, f.lengths, ps,
                                           dy.p, dy.stride, dh, du.data_ptr(), ddt.data_ptr(), f32(da), db.data_ptr(), dc.data_ptr(), f32(dd),
                                           dz.defined() ? dz.data_ptr() : nullptr, f32(dbias), f32(dh0), ws.data_ptr(), (size_t)ws.numel(),
                                           stream_of(a[15], k.dev));
        if (s != SCAN_OK) return status(s);
        PyObject* out = PyDict_New();
        put(out, "du", du);
        put(out, "ddt", ddt);
        put(out, "da", da);
        put(out, "db", db);
        put(out, "dc", dc);
        if (dd.defined()) put(out, "dd", dd);
        if (dz.defined()) put(out, "dz", dz);
        if (dbias.defined()) put(out, "ddt_bias", dbias);
        if (dh0.defined()) put(out, "dh0", dh0);
        return out;
    });
}

// (h, u, dt, a, b, c, d, z, dt_bias, softplus, stream) -> y
LRS_BOUND(ssm_scan_step) {
    return guarded([&]() -> PyObject* {
        need(count == 11);
        const Scan k(a + 1, 2);
        need(a[0] != Py_None);
        float* h = const_cast<float*>(k.state(a[0]));
        Tensor y = empty(k.u.sizes(), k.type, k.dev);
        const scan_status s = ::ssm_scan_step(k.batch, (int)k.d, (int)k.n, (int)k.groups, k.dtype, truth(a[9]), h, k.mu.p, k.mu.stride, k.mdt.p,
                                            k.mdt.stride, k.pa, k.pb, k.sb, k.pc, k.sc, k.skip, k.mz.p, k.mz.stride, k.bias, y.data_ptr(),
                                            stream_of(a[10], k.dev));
        if (s != SCAN_OK) return status(s);
        written(tensor(a[0]));
        return THPVariable_Wrap(y);
    });
}

// (x, w, bias, act, state, reset, lengths, stream) -> (y, state_out)
LRS_BOUND(causal_conv_fwd) {
    return guarded([&]() -> PyObject* {
        need(count == 8);
        const Conv k(a, 3);
        const Flags f(a[5], a[6], k.batch, k.length, k.dev);
        const void* st = k.state(a[4]);
        Tensor y = empty(k.x.sizes(), k.type, k.dev), out = empty({k.batch, k.width - 1, k.d}, k.type, k.dev);
        const scan_status s = ssm_conv_fwd(k.batch, k.length, (int)k.d, (int)k.width, k.dtype, (int)number(a[3]), k.x.data_ptr(), k.stride, k.pw, k.bias,
                                           st, f.reset, f.lengths, y.data_ptr(), out.data_ptr(), stream_of(a[7], k.dev));
        if (s != SCAN_OK) return status(s);
        return Py_BuildValue("(NN)", THPVariable_Wrap(y), THPVariable_Wrap(out));
    });
}

// (x, w, bias, dy, dstate_out, act, state, reset, lengths, stream) -> dict
LRS_BOUND(causal_conv_bwd) {
    return guarded([&]() -> PyObject* {
        need(count == 10);
        const Conv k(a, 3);
        const Flags f(a[7], a[8], k.batch, k.length, k.dev);
        const void *st = k.state(a[6]), *os = k.state(a[4]);
        need(a[3] != Py_None);
        const Matrix dy = matrix(a[3], k.x, k.type);
        const size_t bytes = ssm_conv_bwd_workspace_bytes(k.batch, k.length, (int)k.d, (int)k.width);
        need(bytes > 0);
        Tensor dx = empty(k.x.sizes(), k.type, k.dev), dw = empty({k.d, k.width}, at::kFloat, k.dev), db, ds, ws = empty({(int64_t)bytes}, at::kByte, k.dev);
        if (k.bias) db = empty({k.d}, at::kFloat, k.dev);
        if (a[6] != Py_None) ds = empty({k.batch, k.width - 1, k.d}, k.type, k.dev);
        const scan_status s = ssm_conv_bwd(k.batch, k.length, (int)k.d, (int)k.width, k.dtype, (int)number(a[5]), k.x.data_ptr(), k.stride, k.pw, k.bias,
                                           st, f.reset, f.lengths, dy.p, dy.stride, os, dx.data_ptr(), static_cast<float*>(dw.data_ptr()),
                                           db.defined() ? static_cast<float*>(db.data_ptr()) : nullptr, ds.defined() ? ds.data_ptr() : nullptr,
                                           ws.data_ptr(), bytes, stream_of(a[9], k.dev));
        if (s != SCAN_OK) return status(s);
        PyObject* out = PyDict_New();
        put(out, "dx", dx);
        put(out, "dw", dw);
        if (db.defined()) put(out, "dbias", db);
        if (ds.defined()) put(out, "dstate", ds);
        return out;
    });
}

// (x, w, bias, state, act, stream) -> y
LRS_BOUND(causal_conv_step) {
    return guarded([&]() -> PyObject* {
        need(count == 6);
        const Conv k(a, 2);
        need(a[3] != Py_None);
        void* st = k.state(a[3]);
        Tensor y = empty(k.x.sizes(), k.type, k.dev);
        const scan_status s = ssm_conv_step(k.batch, (int)k.d, (int)k.width, k.dtype, (int)number(a[4]), k.x.data_ptr(), k.stride, k.pw, k.bias, st,
                                            y.data_ptr(), stream_of(a[5], k.dev));
        if (s != SCAN_OK) return status(s);
        written(tensor(a[3]));
        return THPVariable_Wrap(y);
    });
}

}  // namespace lrs_bind
