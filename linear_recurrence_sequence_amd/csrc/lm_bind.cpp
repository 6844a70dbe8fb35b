// lm_bind.cpp -- the usual calls of lm.py without its per-tensor Python work.
//
// A call of a small operator takes a few microseconds on the GPU; reading
// dtype, shape, strides and address of each of its tensors from Python takes
// 0.4 us a tensor, 60 us for an AdamW step over 24 tensors with 8-bit states.
// Here the same checks are made on the C++ tensors.  Each function returns None
// where a call is not plainly right (lm.py then makes its own checks, says what is
// wrong, or handles the rarer layout), the library's status where the library
// refused it, and otherwise the call's results.
#include "lm_bind.hpp"

#include <vector>

#include "lm_ops.h"

using namespace lrs_bind;

namespace {

struct Norm {
    const Tensor& x;
    const Tensor& y;
    c10::Device dev;
    int64_t d, rows;
    int st, br, act;
    Matrix mx, my, mg;
    float *w_post, *scale, *w_pre;
    // a: x, y, gate, w_post, scale, w_pre; act: the gate's code
    Norm(PyObject* const* a, PyObject* act_code)
        : x(tensor(a[0])), y(tensor(a[1])), dev(x.device()), d(0), rows(0) {
        need(dev.is_cuda() && x.dim() >= 1 && x.size(-1) >= 1);
        d = x.size(-1);
        rows = x.numel() / d;
        st = code(x.scalar_type());
        br = code(y.scalar_type());
        act = (int)PyLong_AsLong(act_code);
        mx = matrix(a[0], x, x.scalar_type());
        my = matrix(a[1], x, y.scalar_type());
        mg = matrix(a[2], x, y.scalar_type());
        w_post = vec(a[3], d, dev);
        scale = vec(a[4], d, dev);
        w_pre = vec(a[5], d, dev);
        need(w_pre && (w_post == nullptr) == (scale == nullptr) && (a[2] == Py_None) == (act == 0));
    }
};

// (x, y, gate, w_post, scale, w_pre, eps, act, stream) -> (r, n, stats)
PyObject* block_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        need(count == 9);
        const Norm k(a, a[7]);
        Tensor r = empty(k.x.sizes(), k.x.scalar_type(), k.dev), n = empty(k.x.sizes(), k.y.scalar_type(), k.dev),
               stats = empty({k.rows, 2}, at::kFloat, k.dev);
        const scan_status s = lm_block_norm_fwd(k.rows, (int)k.d, k.st, k.br, k.act, number(a[6]), k.mx.p, k.mx.stride, k.my.p,
                                                k.my.stride, k.mg.p, k.mg.stride, k.w_post, k.scale, k.w_pre, r.data_ptr(),
                                                n.data_ptr(), static_cast<float*>(stats.data_ptr()), stream_of(a[8], k.dev));
        if (s != SCAN_OK) return status(s);
        return Py_BuildValue("(NNN)", THPVariable_Wrap(r), THPVariable_Wrap(n), THPVariable_Wrap(stats));
    });
}

// (x, y, gate, w_post, scale, w_pre, stats, dr, dn, act, stream) -> dict
PyObject* block_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        need(count == 11);
        const Norm k(a, a[9]);
        const Tensor& stats = tensor(a[6]);
        need(stats.dim() == 2 && stats.size(0) == k.rows && stats.size(1) == 2);
        const float* ps = static_cast<const float*>(dense(stats, at::kFloat, k.dev));
        const Matrix dr = matrix(a[7], k.x, k.x.scalar_type()), dn = matrix(a[8], k.x, k.y.scalar_type());
        const size_t bytes = lm_block_norm_bwd_workspace_bytes(k.rows, (int)k.d);
        need(bytes > 0);
        Tensor dx = empty(k.x.sizes(), k.x.scalar_type(), k.dev), dy = empty(k.x.sizes(), k.y.scalar_type(), k.dev), dg;
        if (k.mg.p || a[2] != Py_None) dg = empty(k.x.sizes(), k.y.scalar_type(), k.dev);
        // the three weights' gradients in one allocation
        const int64_t line = (k.d + 63) / 64 * 64;
        Tensor dw = empty({k.w_post ? 3 : 1, line}, at::kFloat, k.dev), ws = empty({(int64_t)bytes}, at::kByte, k.dev);
        float* pw = static_cast<float*>(dw.data_ptr());
        const scan_status s = lm_block_norm_bwd(k.rows, (int)k.d, k.st, k.br, k.act, k.mx.p, k.mx.stride, k.my.p, k.my.stride, k.mg.p,
                                                k.mg.stride, k.w_post, k.scale, k.w_pre, ps, dr.p, dr.stride, dn.p, dn.stride,
                                                dx.data_ptr(), dy.data_ptr(), dg.defined() ? dg.data_ptr() : nullptr,
                                                k.w_post ? pw + line : nullptr, k.w_post ? pw + 2 * line : nullptr, pw, ws.data_ptr(),
                                                bytes, stream_of(a[10], k.dev));
        if (s != SCAN_OK) return status(s);
        PyObject* out = PyDict_New();
        put(out, "dx", dx);
        put(out, "dy", dy);
        if (dg.defined()) put(out, "dgate", dg);
        if (k.w_post) {
            put(out, "dw_post", dw.as_strided({k.d}, {1}, line));
            put(out, "dscale", dw.as_strided({k.d}, {1}, 2 * line));
        }
        put(out, "dw_pre", dw.as_strided({k.d}, {1}, 0));
        return out;
    });
}

struct Head {
    const Tensor& h;
    const Tensor& w;
    const Tensor& target;
    c10::Device dev;
    int64_t n, d, v, stride;
    void *ph, *pw;
    const int64_t* pt;
    explicit Head(PyObject* const* a) : h(tensor(a[0])), w(tensor(a[1])), target(tensor(a[2])), dev(h.device()) {
        need(dev.is_cuda() && h.dim() >= 1 && w.dim() == 2 && h.scalar_type() == at::kBFloat16 && h.size(-1) == w.size(1));
        need(target.sizes() == h.sizes().slice(0, h.dim() - 1));
        n = target.numel(), d = w.size(1), v = w.size(0), stride = row_stride(h);
        ph = h.data_ptr();
        pw = dense(w, at::kBFloat16, dev);
        pt = static_cast<const int64_t*>(dense(target, at::kLong, dev));
    }
    const float* token(PyObject* o, bool optional) const {
        if (optional && o == Py_None) return nullptr;
        const Tensor& t = tensor(o);
        need(t.sizes() == target.sizes());
        return static_cast<const float*>(dense(t, at::kFloat, dev));
    }
    Tensor workspace(int backward) const {
        const size_t bytes = lm_linear_ce_workspace_bytes(n, (int)d, v, backward);
        need(bytes > 0);
        return empty({(int64_t)bytes}, at::kByte, dev);
    }
};

// (h, w, target, softcap, stream) -> (loss, lse)
PyObject* linear_ce_fwd(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        need(count == 5);
        const Head k(a);
        Tensor loss = empty(k.target.sizes(), at::kFloat, k.dev), lse = empty(k.target.sizes(), at::kFloat, k.dev), ws = k.workspace(0);
        const scan_status s = lm_linear_ce_fwd(k.n, (int)k.d, k.v, number(a[3]), k.ph, k.stride, k.pw, k.pt,
                                               static_cast<float*>(loss.data_ptr()), static_cast<float*>(lse.data_ptr()),
                                               ws.data_ptr(), (size_t)ws.numel(), stream_of(a[4], k.dev));
        if (s != SCAN_OK) return status(s);
        return Py_BuildValue("(NN)", THPVariable_Wrap(loss), THPVariable_Wrap(lse));
    });
}

// (h, w, target, lse, dloss, dlse, softcap, gradients in FP32, stream) -> dict
PyObject* linear_ce_bwd(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        need(count == 9);
        const Head k(a);
        const float *lse = k.token(a[3], false), *dloss = k.token(a[4], false), *dlse = k.token(a[5], true);
        const bool f32 = PyObject_IsTrue(a[7]) == 1;
        const at::ScalarType type = f32 ? at::kFloat : at::kBFloat16;
        Tensor dh = empty(k.h.sizes(), type, k.dev), dw = empty(k.w.sizes(), type, k.dev), ws = k.workspace(1);
        const scan_status s = lm_linear_ce_bwd(k.n, (int)k.d, k.v, number(a[6]), k.ph, k.stride, k.pw, k.pt, lse, dloss, dlse,
                                               dh.data_ptr(), dw.data_ptr(), f32 ? SCAN_F32 : SCAN_BF16, ws.data_ptr(),
                                               (size_t)ws.numel(), stream_of(a[8], k.dev));
        if (s != SCAN_OK) return status(s);
        PyObject* out = PyDict_New();
        put(out, "dh", dh);
        put(out, "dw", dw);
        return out;
    });
}

// The addresses of a list of dense tensors of one type with the given sizes.
struct List {
    PyObject* fast = nullptr;
    std::vector<void*> at;
    ~List() { Py_XDECREF(fast); }
    void open(PyObject* o) {
        fast = PySequence_Fast(o, "");
        need(fast != nullptr);
    }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
    const Tensor& operator[](Py_ssize_t i) const { return tensor(PySequence_Fast_GET_ITEM(fast, i)); }
    void read(PyObject* o, const std::vector<int64_t>& n, at::ScalarType type, const c10::Device& dev) {
        if (!fast) open(o);
        need(size() == (Py_ssize_t)n.size());
        at.resize(n.size());
        for (size_t i = 0; i < n.size(); ++i) {
            const Tensor& t = (*this)[(Py_ssize_t)i];
            need(t.numel() == n[i]);
            at[i] = dense(t, type, dev);
        }
    }
    // says to autograd that a call wrote the tensors (5 ns each: of a step's, the weights, which graphs keep)
    void written() const {
        for (Py_ssize_t i = 0; fast && i < size(); ++i)
            lrs_bind::written((*this)[i]);
    }
    template <class T>
    T* const* as() {
        return fast ? reinterpret_cast<T* const*>(at.data()) : nullptr;
    }
};

// (params, grads, m, v, masters, m_scales, v_scales, weight_decay, step, lr, beta1, beta2, eps, stream) -> status
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        need(count == 14);
        List l[7];
        l[0].open(a[0]);
        l[1].open(a[1]);
        const Py_ssize_t k = l[0].size();
        need(k > 0 && l[1].size() == k);
        const c10::Device dev = l[0][0].device();
        need(dev.is_cuda() && (a[5] == Py_None) == (a[6] == Py_None));
        const bool bits8 = a[5] != Py_None;
        std::vector<int64_t> n((size_t)k), blocks((size_t)k);
        std::vector<double> decay((size_t)k);
        for (Py_ssize_t i = 0; i < k; ++i) {
            n[i] = l[0][i].numel();
            blocks[i] = (n[i] + LM_ADAMW_BLOCK - 1) / LM_ADAMW_BLOCK;
        }
        const at::ScalarType pt = l[0][0].scalar_type(), gt = l[1][0].scalar_type(), mt = bits8 ? at::kFloat8_e4m3fn : at::kFloat;
        l[0].read(a[0], n, pt, dev);
        l[1].read(a[1], n, gt, dev);
        l[2].read(a[2], n, mt, dev);
        l[3].read(a[3], n, mt, dev);
        if (a[4] != Py_None) l[4].read(a[4], n, at::kFloat, dev);
        if (bits8) {
            l[5].read(a[5], blocks, at::kFloat, dev);
            l[6].read(a[6], blocks, at::kFloat, dev);
        }
        if (PyList_Check(a[7]) || PyTuple_Check(a[7])) {
            List w;
            w.open(a[7]);
            need(w.size() == k);
            for (Py_ssize_t i = 0; i < k; ++i) decay[i] = number(PySequence_Fast_GET_ITEM(w.fast, i));
        } else {
            decay.assign((size_t)k, number(a[7]));
        }
        const long long step = PyLong_AsLongLong(a[8]);
        need(!PyErr_Occurred());
        const scan_status st = lm_adamw_step((int)k, code(pt), code(gt), bits8 ? 8 : 32, l[0].as<void>(), l[1].as<const void>(),
                                             l[2].as<void>(), l[3].as<void>(), l[4].as<float>(), l[5].as<float>(), l[6].as<float>(),
                                             n.data(), decay.data(), number(a[9]), number(a[10]), number(a[11]), number(a[12]), step, stream_of(a[13], dev));
        if (st == SCAN_OK) l[0].written();
        return status(st);
    });
}

// (tokens, w, scale, out in FP32: True, False or None (as w), stream) -> out
PyObject* embed_fwd(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        need(count == 5);
        const Tensor &t = tensor(a[0]), &w = tensor(a[1]);
        const c10::Device dev = w.device();
        need(dev.is_cuda() && w.dim() == 2 && w.size(0) >= 1 && w.size(1) >= 1);
        const int wt = code(w.scalar_type());
        const int64_t* pt = static_cast<const int64_t*>(dense(t, at::kLong, dev));
        const void* pw = dense(w, w.scalar_type(), dev);
        const at::ScalarType type = a[3] == Py_None ? w.scalar_type() : a[3] == Py_True ? at::kFloat : at::kBFloat16;
        std::vector<int64_t> shape(t.sizes().begin(), t.sizes().end());
        shape.push_back(w.size(1));
        need(w.size(1) <= (1 << 23));
        Tensor out = empty(shape, type, dev);
        const scan_status s = lm_embed_fwd(t.numel(), (int)w.size(1), w.size(0), wt, code(type), number(a[2]), pt, pw, out.data_ptr(), stream_of(a[4], dev));
        if (s != SCAN_OK) return status(s);
        return THPVariable_Wrap(out);
    });
}

// (tokens, dout, v, scale, gradient in FP32, stream) -> dw
PyObject* embed_bwd(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        need(count == 6);
        const Tensor &t = tensor(a[0]), &g = tensor(a[1]);
        const c10::Device dev = g.device();
        need(dev.is_cuda() && g.dim() >= 1 && g.size(-1) >= 1 && g.size(-1) <= (1 << 23) && t.sizes() == g.sizes().slice(0, g.dim() - 1) && PyLong_Check(a[2]));
        const long long v = PyLong_AsLongLong(a[2]);
        need(!PyErr_Occurred() && v >= 1);
        const int64_t d = g.size(-1), n = t.numel(), *pt = static_cast<const int64_t*>(dense(t, at::kLong, dev));
        const int gt = code(g.scalar_type());
        const int64_t stride = row_stride(g);
        const size_t bytes = lm_embed_bwd_workspace_bytes(n, (int)d, v);
        need(bytes > 0);
        const at::ScalarType type = a[4] == Py_True ? at::kFloat : at::kBFloat16;
        Tensor dw = empty({v, d}, type, dev), ws = empty({(int64_t)bytes}, at::kByte, dev);
        const scan_status s = lm_embed_bwd(n, (int)d, v, gt, code(type), number(a[3]), pt, g.data_ptr(), stride, 0, dw.data_ptr(), ws.data_ptr(), bytes,
                                           stream_of(a[5], dev));
        if (s != SCAN_OK) return status(s);
        return THPVariable_Wrap(dw);
    });
}

// (torch's function for the current device, and for the current stream's address of a device)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t count) {
    if (count != 2) {
        PyErr_SetString(PyExc_TypeError, "setup takes two functions");
        return nullptr;
    }
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    current_device = a[0];
    current_stream = a[1];
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(block_norm_fwd), METHOD(block_norm_bwd), METHOD(linear_ce_fwd), METHOD(linear_ce_bwd),
                         METHOD(adamw_step),     METHOD(embed_fwd),      METHOD(embed_bwd),     METHOD(ssm_scan_fwd),
                         METHOD(ssm_scan_bwd),   METHOD(ssm_scan_step),  METHOD(causal_conv_fwd), METHOD(causal_conv_bwd),
                         METHOD(causal_conv_step), METHOD(setup),          {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm_bind() { return PyModule_Create(&module); }
