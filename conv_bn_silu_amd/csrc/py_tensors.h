// py_tensors.h -- what the Python side of the calls shares (py_block8.cpp, py_step.cpp): checks of
// tensors, outputs and workspaces from PyTorch's allocator, the current stream, records of caches.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/cbs_step.h"

namespace cbs_py {

struct Refused {};  // a Python error is set
[[noreturn]] inline void refuse(PyObject *kind, const std::string &why) {
    PyErr_SetString(kind, why.c_str());
    throw Refused();
}

inline int code_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return CBS_DTYPE_F32;
        case at::kBFloat16: return CBS_DTYPE_BF16;
        case at::kHalf: return CBS_DTYPE_F16;
        case at::kChar: return CBS_DTYPE_I8;
        default: return -1;
    }
}
inline const char *name_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kChar: return "torch.int8";
        case at::kInt: return "torch.int32";
        case at::kDouble: return "torch.float64";
        default: return "?";
    }
}
// A call goes to the current device, whose handle and stream it takes.
inline void on_current_device(const at::Tensor &t, const char *what) {
    const int now = c10::hip::current_device(), its = t.device().index();
    if (its != now)
        refuse(PyExc_ValueError, std::string(what) + " is on cuda:" + std::to_string(its) + ", and the current device is cuda:" +
                                     std::to_string(now));
}
using Types = std::initializer_list<at::ScalarType>;
constexpr at::ScalarType kValues[] = {at::kFloat, at::kBFloat16, at::kHalf};
const Types kValueTypes = {at::kFloat, at::kBFloat16, at::kHalf};

inline const at::Tensor &tensor(PyObject *o, const char *what, Types types, const at::Tensor *beside = nullptr) {
    const bool is = THPVariable_Check(o);
    bool fits = false;
    if (is)
        for (at::ScalarType t : types) fits |= THPVariable_Unpack(o).scalar_type() == t;
    if (!fits) {
        std::string s = std::string(what) + " must be a tensor of type ";
        for (at::ScalarType t : types) s += std::string(t == *types.begin() ? "" : " or ") + name_of(t);
        refuse(PyExc_TypeError, s);
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.requires_grad() && at::GradMode::is_enabled())
        refuse(PyExc_ValueError, std::string(what) + " requires a gradient: these operators are forward only");
    if (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
        refuse(PyExc_ValueError, std::string(what) + " carries a tangent: these operators are forward only");
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(what) + " must be a device tensor");
    if (beside && t.device() != beside->device()) refuse(PyExc_ValueError, std::string(what) + " is on another device");
    return t;
}
inline void contiguous(const at::Tensor &t, at::IntArrayRef shape, const char *what) {
    if (t.sizes() == shape && t.is_contiguous()) return;
    std::string s = std::string(what) + " must be contiguous, of shape (";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    refuse(PyExc_ValueError, s + ")");
}
inline at::Tensor output(PyObject *out, at::IntArrayRef shape, const at::Tensor &like, const char *what = "out") {
    if (out == Py_None) return at::empty(shape, like.options().requires_grad(false));
    const at::Tensor &t = tensor(out, what, {like.scalar_type()}, &like);
    contiguous(t, shape, what);
    return t;
}
inline at::Tensor workspace(int64_t bytes, const at::Tensor &like) {
    return bytes > 0 ? at::empty({bytes}, like.options().dtype(at::kChar).requires_grad(false)) : at::Tensor();
}
inline void *data(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
inline void *stream(const at::Tensor &t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }
inline int64_t bytes_of(int64_t n) { return n > 0 ? n : 0; }

inline conv_bn_silu_t handle(PyObject *o) {
    if (o == Py_None) return nullptr;
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused();
    return (conv_bn_silu_t)p;
}
inline long whole(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
inline PyObject *result(int status, const at::Tensor &y) { return status == CBS_OK ? THPVariable_Wrap(y) : PyLong_FromLong(status); }

template <typename F> inline PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F &&f) {
    HANDLE_TH_ERRORS
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// A cache's record, in a capsule: the tensors, and their addresses as the C ABI takes them.
struct Record {
    cbs_paged_cache c;
    at::Tensor k, v, k_scale, v_scale;
    int64_t elements;
    // The tensors' memory may be exchanged under the record (set_, resize_, an assignment to .data).
    bool holds() const {
        if (k.data_ptr() != c.k || v.data_ptr() != c.v || k.numel() != elements || v.numel() != elements) return false;
        if (!k_scale.defined()) return true;
        return k_scale.data_ptr() == c.k_scale && v_scale.data_ptr() == c.v_scale && k_scale.numel() * c.dim == elements &&
               v_scale.numel() * c.dim == elements;
    }
};
constexpr const char *kCapsule = "conv_bn_silu_amd.cache";
inline const Record &record(PyObject *o) {
    const Record *r = (const Record *)PyCapsule_GetPointer(o, kCapsule);
    if (!r) throw Refused();
    on_current_device(r->k, "the cache");
    if (!r->holds()) refuse(PyExc_ValueError, "the cache's tensors have been given other memory: make a PagedCache of them");
    return *r;
}

inline const at::Tensor &slots_of(PyObject *o, const at::Tensor &cache, int64_t tokens) {
    const at::Tensor &s = tensor(o, "slots", {at::kInt}, &cache);
    if (s.dim() != 1 || !s.is_contiguous() || (tokens >= 0 && s.size(0) != tokens))
        refuse(PyExc_ValueError, "slots must be contiguous, one for each token");
    return s;
}

// The methods of py_step.cpp, ended by an empty one.
extern PyMethodDef step_methods[];

}  // namespace cbs_py
