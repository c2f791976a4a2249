// py_step.cpp -- the Python side of include/cbs_step.h's calls and of the linear layer on
// rows in 8 bits; as in py_block8.cpp, each function returns its result or a status.
#include "py_tensors.h"

namespace {

using namespace cbs_py;

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}
at::ScalarType value_dtype(PyObject *o, const char *what) {
    if (THPDtype_Check(o)) {
        const at::ScalarType type = reinterpret_cast<THPDtype *>(o)->scalar_type;
        for (at::ScalarType t : kValues)
            if (t == type) return type;
    }
    refuse(PyExc_TypeError, std::string(what) + " must be float32, bfloat16 or float16");
}

// [..., K] as rows that the kernels take; copied where its rows are not contiguous.
at::Tensor rows_of(const at::Tensor &x, int64_t K) {
    at::Tensor rows = x.dim() == 2 ? x : x.reshape({-1, K});
    if ((K > 1 && rows.stride(1) != 1) || (rows.size(0) > 1 && rows.stride(0) < K)) rows = rows.contiguous();
    return rows;
}
int64_t stride_of(const at::Tensor &rows, int64_t K) { return rows.size(0) > 1 ? rows.stride(0) : K; }

// (handle, x, weight, residual, eps, int8, out, sum_out) -> y, or (y, sum); for int8 y is the buffer of the rows
PyObject *add_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[1], "x", kValueTypes);
        on_current_device(x, "x");
        if (x.dim() < 1 || x.size(-1) < 1) refuse(PyExc_ValueError, "x must be [..., K] with K of 1 or more");
        const int64_t K = x.size(-1);
        const at::Tensor rows = rows_of(x, K);
        const int64_t M = rows.size(0);
        const void *weight = nullptr;
        int weight_type = CBS_DTYPE_F32;
        if (a[2] != Py_None) {
            const at::Tensor &w = tensor(a[2], "weight", {x.scalar_type(), at::kFloat}, &x);
            contiguous(w, {K}, "weight");
            weight = w.data_ptr(), weight_type = code_of(w.scalar_type());
        }
        const double eps = number(a[4]);
        if (!((float)eps >= 0x1p-126f) || !std::isfinite((float)eps)) refuse(PyExc_ValueError, "eps must be 2^-126 or more, and finite");
        const bool int8 = truth(a[5]);
        at::Tensor residual, sum;
        if (a[3] != Py_None) {
            const at::Tensor &r = tensor(a[3], "residual", {x.scalar_type(), at::kFloat}, &x);
            if (r.sizes() != x.sizes()) refuse(PyExc_ValueError, "residual must have the shape of x");
            sum = output(a[7], x.sizes(), r, "sum_out");
            residual = rows_of(r, K);
        } else if (a[7] != Py_None) {
            refuse(PyExc_ValueError, "sum_out needs a residual");
        }
        at::Tensor y;
        if (int8) {
            if (a[6] != Py_None) refuse(PyExc_ValueError, "rows in 8 bits take no out");
            const int64_t bytes = cbs_rows8_bytes(M, K);
            y = at::empty({bytes_of(bytes)}, x.options().dtype(at::kChar).requires_grad(false));
        } else {
            y = output(a[6], x.sizes(), x);
        }
        const int status = cbs_add_rms_norm(
            handle(a[0]), rows.data_ptr(), stride_of(rows, K), data(residual), residual.defined() ? stride_of(residual, K) : K,
            code_of(residual.defined() ? residual.scalar_type() : x.scalar_type()), weight, weight_type, (float)eps, data(sum), K,
            y.data_ptr(), int8 ? (int)CBS_DTYPE_I8 : code_of(x.scalar_type()), M, K, code_of(x.scalar_type()), stream(x));
        if (status != CBS_OK) return PyLong_FromLong(status);
        PyObject *py = THPVariable_Wrap(y);
        if (!sum.defined() || !py) return py;
        PyObject *ps = a[7] == Py_None ? THPVariable_Wrap(sum) : Py_NewRef(a[7]);
        PyObject *both = ps ? PyTuple_Pack(2, py, ps) : nullptr;
        Py_DECREF(py);
        Py_XDECREF(ps);
        return both;
    });
}

// (handle, buffer, shape, dtype, w, w_scale, bias, activation, out)
PyObject *int8_linear_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const at::Tensor &rows = tensor(a[1], "rows", {at::kChar});
        on_current_device(rows, "rows");
        if (!PyTuple_Check(a[2]) || PyTuple_GET_SIZE(a[2]) < 1) refuse(PyExc_TypeError, "the rows' shape must be a tuple, [..., K]");
        c10::SmallVector<int64_t, 8> shape;
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[2]); ++i) shape.push_back(whole(PyTuple_GET_ITEM(a[2], i)));
        const int64_t K = shape.back();
        int64_t M = 1;
        for (size_t i = 0; i + 1 < shape.size(); ++i) {
            if (shape[i] < 0 || (shape[i] > 0 && M > INT32_MAX / shape[i])) refuse(PyExc_ValueError, "the rows' shape cannot be");
            M *= shape[i];
        }
        const at::ScalarType type = value_dtype(a[3], "dtype");
        const at::Tensor &w = tensor(a[4], "w", {at::kChar}, &rows);
        const at::Tensor &ws = tensor(a[5], "w_scale", {at::kFloat}, &rows);
        if (w.dim() != 2 || w.size(1) != K) refuse(PyExc_ValueError, "x must be [..., K] and w [N, K]");
        const int act = (int)whole(a[7]);
        if (act < 0) refuse(PyExc_ValueError, "activation must be None or 'silu'");
        const int64_t N = w.size(0);
        contiguous(w, {N, K}, "w");
        contiguous(ws, {N}, "w_scale");
        contiguous(rows, {bytes_of(cbs_rows8_bytes(M, K))}, "rows");
        const void *bias = nullptr;
        if (a[6] != Py_None) {
            const at::Tensor &b = tensor(a[6], "bias", {at::kFloat}, &rows);
            contiguous(b, {N}, "bias");
            bias = b.data_ptr();
        }
        shape.back() = N;
        at::Tensor y;
        if (a[8] == Py_None) {
            y = at::empty(shape, rows.options().dtype(type).requires_grad(false));
        } else {
            y = tensor(a[8], "out", {type}, &rows);
            contiguous(y, shape, "out");
        }
        const int64_t need = cbs_int8_linear_rows_workspace(M, N, K);
        const at::Tensor tmp = workspace(need, rows);
        return result(cbs_int8_linear_rows(handle(a[0]), rows.data_ptr(), (const int8_t *)w.data_ptr(), (const float *)ws.data_ptr(),
                                           (const float *)bias, y.data_ptr(), M, N, K, code_of(type), act, data(tmp), bytes_of(need),
                                           stream(rows)),
                      y);
    });
}

// [tokens, heads, dim] with dim contiguous.
const at::Tensor &heads_of(PyObject *o, const char *what, Types types, const at::Tensor *beside) {
    const at::Tensor &t = tensor(o, what, types, beside);
    if (t.dim() != 3 || (t.size(2) > 1 && t.stride(2) != 1))
        refuse(PyExc_ValueError, std::string(what) + " must be [tokens, heads, dim] with dim contiguous");
    if (t.size(1) > INT32_MAX || t.size(2) > INT32_MAX) refuse(PyExc_ValueError, std::string(what) + " is too large");
    return t;
}
const int32_t *per_token(PyObject *o, const char *what, const at::Tensor &beside, int64_t tokens) {
    const at::Tensor &t = tensor(o, what, {at::kInt}, &beside);
    if (t.dim() != 1 || t.size(0) != tokens || !t.is_contiguous())
        refuse(PyExc_ValueError, std::string(what) + " must be contiguous, one for each token");
    return (const int32_t *)t.data_ptr();
}
cbs_rotary rotary_of(PyObject *frequencies, PyObject *interleaved, PyObject *magnitude, const at::Tensor &beside, int64_t dim) {
    const at::Tensor &f = tensor(frequencies, "frequencies", {at::kDouble}, &beside);
    if (f.dim() != 1 || f.size(0) < 1 || !f.is_contiguous() || 2 * f.size(0) > dim)
        refuse(PyExc_ValueError, "frequencies must be contiguous, one for each pair of dims, " + std::to_string(dim / 2) + " at most");
    const double m = number(magnitude);
    if (!std::isfinite((float)m)) refuse(PyExc_ValueError, "magnitude must be finite");
    return cbs_rotary{(const double *)f.data_ptr(), (int32_t)f.size(0), truth(interleaved), (float)m};
}
at::Tensor heads_out(PyObject *out, const at::Tensor &x) {
    if (out == Py_None) return at::empty(x.sizes(), x.options().requires_grad(false));
    const at::Tensor &t = heads_of(out, "out", {x.scalar_type()}, &x);
    if (t.sizes() != x.sizes()) refuse(PyExc_ValueError, "out must have the shape of the input");
    return t;
}

// (handle, x, positions, frequencies, interleaved, magnitude, out)
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const at::Tensor &x = heads_of(a[1], "x", kValueTypes, nullptr);
        on_current_device(x, "x");
        if (x.size(1) < 1) refuse(PyExc_ValueError, "x has no heads");
        const cbs_rotary r = rotary_of(a[3], a[4], a[5], x, x.size(2));
        const int32_t *positions = per_token(a[2], "positions", x, x.size(0));
        const at::Tensor y = heads_out(a[6], x);
        return result(cbs_rotary_apply(handle(a[0]), &r, x.data_ptr(), x.stride(0), x.stride(1), positions, x.size(0),
                                       (int)x.size(1), (int)x.size(2), code_of(x.scalar_type()), y.data_ptr(), y.stride(0),
                                       y.stride(1), stream(x)),
                      y);
    });
}

// (handle, cache, q, k, v, positions, slots, frequencies, interleaved, magnitude, out)
PyObject *rotary_cache_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        const Record &c = record(a[1]);
        const at::Tensor &q = heads_of(a[2], "q", kValueTypes, &c.k);
        const at::Tensor &k = heads_of(a[3], "k", {q.scalar_type()}, &c.k);
        const at::Tensor &v = heads_of(a[4], "v", {q.scalar_type()}, &c.k);
        if (q.size(2) != c.c.dim) refuse(PyExc_ValueError, "q must be [tokens, heads, " + std::to_string(c.c.dim) + "]");
        const int64_t tokens = q.size(0);
        for (const at::Tensor *t : {&k, &v})
            if (t->size(0) != tokens || t->size(1) != c.c.heads || t->size(2) != c.c.dim)
                refuse(PyExc_ValueError, std::string(t == &k ? "k" : "v") + " must be [tokens, " + std::to_string(c.c.heads) +
                                             ", " + std::to_string(c.c.dim) + "]");
        const cbs_rotary r = rotary_of(a[7], a[8], a[9], c.k, c.c.dim);
        const int32_t *positions = per_token(a[5], "positions", c.k, tokens), *slots = per_token(a[6], "slots", c.k, tokens);
        const at::Tensor y = heads_out(a[10], q);
        return result(cbs_rotary_cache_write(handle(a[0]), &r, &c.c, q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(),
                                             k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), positions, slots,
                                             tokens, (int)q.size(1), code_of(q.scalar_type()), y.data_ptr(), y.stride(0),
                                             y.stride(1), stream(c.k)),
                      y);
    });
}

// A pool's record, in a capsule, as a cache's.
struct Pool {
    cbs_page_pool p;
    at::Tensor free, counts;
    bool holds() const {
        return free.data_ptr() == p.free && counts.data_ptr() == p.counts && free.numel() == p.pages && counts.numel() == 3;
    }
};
constexpr const char *kPool = "conv_bn_silu_amd.pool";
const Pool &pool_of(PyObject *o) {
    const Pool *p = (const Pool *)PyCapsule_GetPointer(o, kPool);
    if (!p) throw Refused();
    on_current_device(p->free, "the pool");
    if (!p->holds()) refuse(PyExc_ValueError, "the pool's tensors have been given other memory: make a PagePool of them");
    return *p;
}
// (free, counts, page_size) -> capsule
PyObject *pool(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject * {
        const at::Tensor &free = tensor(a[0], "free", {at::kInt});
        const at::Tensor &counts = tensor(a[1], "counts", {at::kInt}, &free);
        if (free.dim() != 1 || free.size(0) < 1 || !free.is_contiguous()) refuse(PyExc_ValueError, "free must be contiguous, one for each page");
        contiguous(counts, {3}, "counts");
        const long page_size = whole(a[2]);
        if (page_size < 1 || free.size(0) > INT32_MAX || page_size > INT32_MAX / free.size(0))
            refuse(PyExc_ValueError, "page_size must be 1 or more, and all pages below 2^31 slots");
        Pool *p = new Pool{{(int32_t *)free.data_ptr(), (int32_t *)counts.data_ptr(), free.size(0), (int32_t)page_size}, free, counts};
        PyObject *c = PyCapsule_New(p, kPool, [](PyObject *o) { delete (Pool *)PyCapsule_GetPointer(o, kPool); });
        if (!c) delete p;
        return c;
    });
}

struct Sequences {
    int32_t *table, *lens, *change;
    int64_t batch, width, stride;
    Sequences(PyObject *t, PyObject *l, PyObject *c, const char *what, const at::Tensor &beside) {
        const at::Tensor &tab = tensor(t, "table", {at::kInt}, &beside);
        if (tab.dim() != 2 || (tab.size(1) > 1 && tab.stride(1) != 1) || (tab.size(0) > 1 && tab.stride(0) < tab.size(1)))
            refuse(PyExc_ValueError, "table must be [batch, width] with contiguous rows");
        batch = tab.size(0), width = tab.size(1), stride = batch > 1 ? tab.stride(0) : width;
        const at::Tensor &len = tensor(l, "lens", {at::kInt}, &beside);
        const at::Tensor &cha = tensor(c, what, {at::kInt}, &beside);
        contiguous(len, {batch}, "lens");
        contiguous(cha, {batch}, what);
        table = (int32_t *)tab.data_ptr(), lens = (int32_t *)len.data_ptr(), change = (int32_t *)cha.data_ptr();
    }
};

// n elements of a contiguous tensor from `first` on, as a tensor over the same storage.
at::Tensor part_of(const at::Tensor &t, int64_t first, int64_t n) {
    at::Tensor part = at::detail::make_tensor<at::TensorImpl>(c10::Storage(t.storage()), t.key_set(), t.dtype());
    part.unsafeGetTensorImpl()->set_storage_offset(first);
    part.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return part;
}

// (handle, pool, table, lens, more, tokens) -> (starts, slots, positions)
PyObject *grow_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject * {
        const Pool &p = pool_of(a[1]);
        const Sequences s(a[2], a[3], a[4], "more", p.free);
        const int64_t tokens = whole(a[5]);
        if (tokens < 0 || tokens > (1 << 30)) refuse(PyExc_ValueError, "tokens must not be negative, and 2^30 at most");
        // one allocation for the three, which costs the host a fifth less of the call
        const int64_t at_slots = (s.batch + 4) / 4 * 4, at_positions = at_slots + (tokens + 3) / 4 * 4;
        const at::Tensor all_three = at::empty({at_positions + tokens}, p.free.options().requires_grad(false));
        const at::Tensor starts = part_of(all_three, 0, s.batch + 1), slots = part_of(all_three, at_slots, tokens);
        const at::Tensor positions = part_of(all_three, at_positions, tokens);
        const int64_t need = cbs_grow_pages_workspace(s.batch, tokens);
        const at::Tensor tmp = workspace(need, p.free);
        const int status = cbs_grow_pages(handle(a[0]), &p.p, s.table, s.stride, s.width, s.lens, s.change, s.batch, tokens,
                                          (int32_t *)starts.data_ptr(), (int32_t *)slots.data_ptr(), (int32_t *)positions.data_ptr(),
                                          data(tmp), bytes_of(need), stream(p.free));
        if (status != CBS_OK) return PyLong_FromLong(status);
        PyObject *got[3] = {THPVariable_Wrap(starts), THPVariable_Wrap(slots), THPVariable_Wrap(positions)};
        PyObject *all = got[0] && got[1] && got[2] ? PyTuple_Pack(3, got[0], got[1], got[2]) : nullptr;
        for (PyObject *o : got) Py_XDECREF(o);
        return all;
    });
}

// (handle, pool, table, lens, keep) -> None
PyObject *release_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject * {
        const Pool &p = pool_of(a[1]);
        const Sequences s(a[2], a[3], a[4], "keep", p.free);
        const int64_t need = cbs_release_pages_workspace(s.batch, s.width);
        const at::Tensor tmp = workspace(need, p.free);
        const int status = cbs_release_pages(handle(a[0]), &p.p, s.table, s.stride, s.width, s.lens, s.change, s.batch, data(tmp),
                                             bytes_of(need), stream(p.free));
        if (status != CBS_OK) return PyLong_FromLong(status);
        Py_RETURN_NONE;
    });
}

}  // namespace

#define CBS_METHOD(f) {#f, (PyCFunction)(void *)f, METH_FASTCALL, nullptr}
PyMethodDef cbs_py::step_methods[] = {CBS_METHOD(add_rms_norm), CBS_METHOD(int8_linear_rows), CBS_METHOD(rotary),
                                      CBS_METHOD(rotary_cache_write), CBS_METHOD(pool), CBS_METHOD(grow_pages),
                                      CBS_METHOD(release_pages), {nullptr, nullptr, 0, nullptr}};
