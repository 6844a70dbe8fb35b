// lm_bind.hpp -- what the quick calls of lm_bind.cpp and ssm_bind.cpp share:
// checks of C++ tensors that leave a call to Python where it is not plainly
// right.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/as_strided.h>
#include <ATen/ops/empty.h>
#include <c10/core/ScalarType.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "samu_scan.h"

namespace lrs_bind {

using at::Tensor;

// Thrown where the call is left to lm.py.
struct Leave {};

inline void need(bool ok) {
    if (!ok) throw Leave{};
}

inline const Tensor& tensor(PyObject* o) {
    need(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

inline int code(at::ScalarType t) {
    need(t == at::kBFloat16 || t == at::kFloat);
    return t == at::kFloat ? SCAN_F32 : SCAN_BF16;
}

// Address of a dense device tensor of a type on `dev`.
inline void* dense(const Tensor& t, at::ScalarType type, const c10::Device& dev) {
    need(t.scalar_type() == type && t.device() == dev && t.is_contiguous());
    return t.data_ptr();
}

// Elements from one row of t [..., d] to the next: rows of dense columns at one distance.
inline int64_t row_stride(const Tensor& t) {
    const int64_t d = t.size(-1);
    if (t.is_contiguous()) return d;
    need(t.stride(-1) == 1 || d == 1);
    int64_t step = -1, reach = 0;
    for (int64_t i = t.dim() - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (step < 0) step = t.stride(i);
        else need(t.stride(i) == reach);
        reach = t.stride(i) * t.size(i);
    }
    return step < 0 ? d : step;
}

struct Matrix {
    void* p = nullptr;
    int64_t stride = 0;
};
inline Matrix matrix(PyObject* o, const Tensor& like, at::ScalarType type) {
    if (o == Py_None) return {};
    const Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.device() == like.device() && t.sizes() == like.sizes());
    return {t.data_ptr(), row_stride(t)};
}

inline float* vec(PyObject* o, int64_t d, const c10::Device& dev) {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o);
    need(t.dim() == 1 && t.size(0) == d);
    return static_cast<float*>(dense(t, at::kFloat, dev));
}

inline Tensor empty(at::IntArrayRef shape, at::ScalarType type, const c10::Device& dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// The stream given, or the current one; tensors of another device than the current one are left to lm.py.
inline PyObject *current_device, *current_stream;  // torch's own, set by setup
inline void* stream_of(PyObject* o, const c10::Device& dev) {
    PyObject* device = PyObject_CallNoArgs(current_device);
    need(device != nullptr);
    bool here = PyLong_AsLong(device) == dev.index();
    if (here && o != Py_None) {  // a stream of the same device
        PyObject* index = PyObject_GetAttrString(o, "device_index");
        here = index && PyLong_AsLong(index) == dev.index();
        Py_XDECREF(index);
    }
    PyObject* raw = !here ? nullptr : o == Py_None ? PyObject_CallOneArg(current_stream, device) : PyObject_GetAttrString(o, "cuda_stream");
    Py_DECREF(device);
    need(raw != nullptr);
    void* s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    need(!PyErr_Occurred());
    return s;
}
inline double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    need(!PyErr_Occurred());
    return v;
}

// Runs f, which returns a new reference; no C++ exception crosses into Python.
template <class F>
PyObject* guarded(F f) {
    HANDLE_TH_ERRORS
    at::AutoDispatchBelowADInplaceOrView below;  // what is made here has no gradient of its own
    try {
        return f();
    } catch (const Leave&) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    END_HANDLE_TH_ERRORS
}

inline PyObject* status(scan_status st) { return PyLong_FromLong(st); }


inline void put(PyObject* dict, const char* key, const Tensor& t) {
    PyObject* o = THPVariable_Wrap(t);
    PyDict_SetItemString(dict, key, o);
    Py_DECREF(o);
}

// Says to autograd that a call wrote a tensor of the caller's.
inline void written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

#define LRS_BOUND(name) PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t count)
LRS_BOUND(ssm_scan_fwd);
LRS_BOUND(ssm_scan_bwd);
LRS_BOUND(ssm_scan_step);
LRS_BOUND(causal_conv_fwd);
LRS_BOUND(causal_conv_bwd);
LRS_BOUND(causal_conv_step);

}  // namespace lrs_bind
