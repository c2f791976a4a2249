// py_block8.cpp -- the Python side of the 8-bit block operators' calls: checks of the
// tensors, outputs and workspaces from PyTorch's allocator, the current stream, and the
// call of the C ABI (include/cbs_block8.h).  A serving step makes hundreds of such
// calls, most of a few microseconds on the GPU; marshalled in Python each took 15 to 20
// on the host.
//
// Each function returns its result, or a status of the C ABI as a Python int
// where that refused the call; what the tensors are refused for is raised here.
#include "py_tensors.h"

namespace {

using namespace cbs_py;

// (handle, x, w, w_scale, bias, activation, out)
PyObject *int8_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[1], "x", kValueTypes);
        on_current_device(x, "x");
        const at::Tensor &w = tensor(a[2], "w", {at::kChar}, &x);
        const at::Tensor &ws = tensor(a[3], "w_scale", {at::kFloat}, &x);
        if (x.dim() < 1 || w.dim() != 2 || x.size(-1) != w.size(1)) refuse(PyExc_ValueError, "x must be [..., K] and w [N, K]");
        const int act = (int)whole(a[5]);
        if (act < 0) refuse(PyExc_ValueError, "activation must be None or 'silu'");
        const int64_t N = w.size(0), K = w.size(1);
        contiguous(w, {N, K}, "w");
        contiguous(ws, {N}, "w_scale");
        const void *bias = nullptr;
        if (a[4] != Py_None) {
            const at::Tensor &b = tensor(a[4], "bias", {at::kFloat}, &x);
            contiguous(b, {N}, "bias");
            bias = b.data_ptr();
        }
        at::Tensor rows = x.dim() == 2 ? x : x.reshape({-1, K});
        const int64_t M = rows.size(0);
        if ((K > 1 && rows.stride(1) != 1) || (M > 1 && rows.stride(0) < K)) rows = rows.contiguous();
        c10::SmallVector<int64_t, 8> shape(x.sizes().begin(), x.sizes().end());
        shape.back() = N;
        const at::Tensor y = output(a[6], shape, x);
        const int64_t need = cbs_int8_linear_workspace(M, N, K);
        const at::Tensor tmp = workspace(need, x);
        return result(cbs_int8_linear(handle(a[0]), rows.data_ptr(), M > 1 ? rows.stride(0) : K, (const int8_t *)w.data_ptr(),
                                      (const float *)ws.data_ptr(), (const float *)bias, y.data_ptr(), M, N, K,
                                      code_of(x.scalar_type()), act, data(tmp), bytes_of(need), stream(x)),
                      y);
    });
}

// (k, v, k_scale, v_scale) -> capsule
PyObject *cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject * {
        const at::Tensor &k = tensor(a[0], "k", {at::kFloat, at::kBFloat16, at::kHalf, at::kChar});
        const at::Tensor &v = tensor(a[1], "v", {k.scalar_type()}, &k);
        if (k.dim() != 4) refuse(PyExc_ValueError, "k must be [pages, heads, page_size, dim]");
        contiguous(k, k.sizes(), "k");
        contiguous(v, k.sizes(), "v");
        at::Tensor scales[2];
        if (k.scalar_type() == at::kChar) {
            for (int i = 0; i < 2; ++i) {
                const char *what = i ? "v_scale" : "k_scale";
                const at::Tensor &s = tensor(a[2 + i], what, {at::kFloat}, &k);
                contiguous(s, k.sizes().slice(0, 3), what);
                scales[i] = s;
            }
        } else if (a[2] != Py_None || a[3] != Py_None) {
            refuse(PyExc_ValueError, "only an int8 cache has scales");
        }
        for (int i = 1; i < 4; ++i)
            if (k.size(i) > INT32_MAX) refuse(PyExc_ValueError, "k must be [pages, heads, page_size, dim]");
        Record *r = new Record{{k.data_ptr(), v.data_ptr(), (float *)data(scales[0]), (float *)data(scales[1]), k.size(0),
                                (int32_t)k.size(1), (int32_t)k.size(2), (int32_t)k.size(3), code_of(k.scalar_type())},
                               k, v, scales[0], scales[1], k.numel()};
        PyObject *c = PyCapsule_New(r, kCapsule, [](PyObject *o) { delete (Record *)PyCapsule_GetPointer(o, kCapsule); });
        if (!c) delete r;
        return c;
    });
}

// (handle, cache, k, v, slots) -> None
PyObject *cache_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject * {
        const Record &r = record(a[1]);
        const at::Tensor &k = tensor(a[2], "k", kValueTypes, &r.k);
        const at::Tensor &v = tensor(a[3], "v", {k.scalar_type()}, &r.k);
        for (const at::Tensor *t : {&k, &v})
            if (t->dim() != 3 || t->size(0) != k.size(0) || t->size(1) != r.c.heads || t->size(2) != r.c.dim ||
                (r.c.dim > 1 && t->stride(2) != 1))
                refuse(PyExc_ValueError, std::string(t == &k ? "k" : "v") + " must be [tokens, " + std::to_string(r.c.heads) +
                                             ", " + std::to_string(r.c.dim) + "] with dim contiguous");
        const int64_t tokens = k.size(0);
        const at::Tensor &slots = slots_of(a[4], r.k, tokens);
        const int status = cbs_cache_write(handle(a[0]), &r.c, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                                           v.stride(0), v.stride(1), (const int32_t *)slots.data_ptr(), tokens,
                                           code_of(k.scalar_type()), stream(r.k));
        if (status != CBS_OK) return PyLong_FromLong(status);
        Py_RETURN_NONE;
    });
}

// (handle, cache, slots, dtype) -> (k, v)
PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject * {
        const Record &r = record(a[1]);
        const at::Tensor &slots = slots_of(a[2], r.k, -1);
        bool fits = false;
        at::ScalarType type = at::kFloat;
        if (THPDtype_Check(a[3])) {
            type = reinterpret_cast<THPDtype *>(a[3])->scalar_type;
            for (at::ScalarType t : kValues) fits |= t == type;
        }
        if (!fits) refuse(PyExc_TypeError, "dtype must be float32, bfloat16 or float16");
        const int64_t tokens = slots.size(0);
        const auto options = r.k.options().dtype(type).requires_grad(false);
        const at::Tensor k = at::empty({tokens, r.c.heads, r.c.dim}, options);
        const at::Tensor v = at::empty({tokens, r.c.heads, r.c.dim}, options);
        const int status = cbs_cache_read(handle(a[0]), &r.c, (const int32_t *)slots.data_ptr(), tokens, k.data_ptr(),
                                          v.data_ptr(), code_of(type), stream(r.k));
        if (status != CBS_OK) return PyLong_FromLong(status);
        PyObject *pk = THPVariable_Wrap(k), *pv = THPVariable_Wrap(v);
        PyObject *both = pk && pv ? PyTuple_Pack(2, pk, pv) : nullptr;
        Py_XDECREF(pk);
        Py_XDECREF(pv);
        return both;
    });
}

// (handle, q, cache, table, starts, lens, window, scale, out); scale a float or None
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const at::Tensor &q = tensor(a[1], "q", {at::kBFloat16, at::kHalf});
        on_current_device(q, "q");
        const Record &r = record(a[2]);
        if (r.k.scalar_type() != at::kChar && r.k.scalar_type() != q.scalar_type())
            refuse(PyExc_TypeError, "the cache must be int8 or of q's type");
        if (q.dim() != 3 || q.size(2) != r.c.dim || r.c.heads < 1 || q.size(1) % r.c.heads || q.size(1) == 0 || q.stride(2) != 1)
            refuse(PyExc_ValueError, "q must be [tokens, a multiple of " + std::to_string(r.c.heads) + ", " +
                                         std::to_string(r.c.dim) + "] with dim contiguous");
        const at::Tensor &table = tensor(a[3], "table", {at::kInt}, &q);
        const at::Tensor &starts = tensor(a[4], "starts", {at::kInt}, &q);
        const at::Tensor &lens = tensor(a[5], "lens", {at::kInt}, &q);
        if (table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
            refuse(PyExc_ValueError, "table must be [batch, width] with contiguous rows");
        const int64_t batch = table.size(0), width = table.size(1), tokens = q.size(0), heads = q.size(1);
        contiguous(starts, {batch + 1}, "starts");
        contiguous(lens, {batch}, "lens");
        const long window = whole(a[6]);
        if (window < 0 || window > INT32_MAX) refuse(PyExc_ValueError, "window must not be negative, and below 2^31");
        if (heads > INT32_MAX) refuse(PyExc_ValueError, "too many heads");
        double scale = 1 / std::sqrt((double)r.c.dim);
        if (a[7] != Py_None) {
            scale = PyFloat_AsDouble(a[7]);
            if (scale == -1.0 && PyErr_Occurred()) throw Refused();
        }
        const at::Tensor y = output(a[8], q.sizes(), q);
        const conv_bn_silu_t h = handle(a[0]);
        const int64_t need = cbs_paged_attention_workspace(h, batch, tokens, (int)heads, r.c.heads, r.c.dim, r.c.page_size, width);
        const at::Tensor tmp = workspace(need, q);
        return result(cbs_paged_attention(h, q.data_ptr(), q.stride(0), q.stride(1), &r.c, (const int32_t *)table.data_ptr(),
                                          batch > 1 ? table.stride(0) : width, width, (const int32_t *)starts.data_ptr(),
                                          (const int32_t *)lens.data_ptr(), batch, tokens, (int)heads, (int)window, (float)scale,
                                          y.data_ptr(), code_of(q.scalar_type()), data(tmp), bytes_of(need), stream(q)),
                      y);
    });
}

#define CBS_METHOD(f) {#f, (PyCFunction)(void *)f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CBS_METHOD(int8_linear), CBS_METHOD(cache), CBS_METHOD(cache_write), CBS_METHOD(cache_read),
                         CBS_METHOD(paged_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block8", "Calls of the 8-bit block operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block8() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddFunctions(m, cbs_py::step_methods) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
