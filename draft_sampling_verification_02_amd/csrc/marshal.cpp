// marshal.cpp -- the short way from torch tensors to the cache and attention
// entry points, for calls whose kernels take a few microseconds.
//
// Each function checks its tensors (types, shapes, layouts, one device, which
// is the current one), calls the C entry point on torch's current stream and
// returns its status.  Where anything is not in order it calls nothing and
// returns None: the Python wrapper then takes its own way through the same
// checks, which finds the words.  Nothing is kept between calls.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "dspark.h"

namespace {

struct Entry {
    decltype(&dspark_kv_write) kv_write;
    decltype(&dspark_kv_read) kv_read;
    decltype(&dspark_paged_attention_workspace_size) paged_ws;
    decltype(&dspark_paged_attention) paged;
    decltype(&dspark_prompt_attention_workspace_size) prompt_ws;
    decltype(&dspark_prompt_attention) prompt;
} entry{};
PyObject *raw_stream = nullptr;  // device index -> hipStream_t of torch's current stream
PyObject *current_device = nullptr;

int dtype_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return DSPARK_BF16;
        case at::kHalf: return DSPARK_F16;
        case at::kFloat8_e4m3fn: return DSPARK_E4M3;
        default: return -1;
    }
}

// Collects the tensors of a call; `ok` falls at the first that is not in order.
struct Call {
    bool ok = true;
    int device = -1;

    const at::Tensor *tensor(PyObject *o) {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        const at::Device d = t.device();
        if (!d.is_cuda() || t.layout() != at::kStrided || (device >= 0 && d.index() != device)) {
            ok = false;
            return nullptr;
        }
        device = d.index();
        return &t;
    }
    const at::Tensor *dense(PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
        const at::Tensor *t = tensor(o);
        if (!ok || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return t;
    }
    template <typename P = void>
    P *at_dense(PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
        const at::Tensor *t = dense(o, type, shape);
        return ok ? static_cast<P *>(t->data_ptr()) : nullptr;
    }
    template <typename P = void>
    P *at_dense_or_none(PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
        return o == Py_None ? nullptr : at_dense<P>(o, type, shape);
    }
    // packed rows [n, heads, D] whose heads lie densely in each row
    const at::Tensor *rows(PyObject *o, int64_t &stride) {
        const at::Tensor *t = tensor(o);
        if (!ok || t->dim() != 3) {
            ok = false;
            return nullptr;
        }
        const int64_t n = t->size(0), h = t->size(1), d = t->size(2);
        if (n == 0 || t->stride(2) != 1 || (t->stride(1) != d && h > 1)) ok = false;
        stride = n > 1 ? t->stride(0) : h * d;
        return t;
    }
    // the stream to launch on; false where the tensors' device is not the current one
    bool stream(void *&s) {
        if (!ok) return false;
        PyObject *cur = PyObject_CallNoArgs(current_device);
        const long dev = cur ? PyLong_AsLong(cur) : -1;
        Py_XDECREF(cur);
        if (dev != device) {
            PyErr_Clear();
            return ok = false;
        }
        PyObject *index = PyLong_FromLong(device);
        PyObject *raw = index ? PyObject_CallOneArg(raw_stream, index) : nullptr;
        Py_XDECREF(index);
        if (!raw) {
            PyErr_Clear();
            return ok = false;
        }
        s = PyLong_AsVoidPtr(raw);
        Py_DECREF(raw);
        return ok;
    }
};

struct Cache {
    const at::Tensor *k = nullptr, *v = nullptr;
    uint8_t *k_scale = nullptr, *v_scale = nullptr;
    int dtype = -1, n_pages = 0, heads = 0, page_size = 0, D = 0;
};
bool fits_int(int64_t x) { return x >= 0 && x <= INT32_MAX; }

Cache cache_of(Call &c, PyObject *k, PyObject *v, PyObject *ks, PyObject *vs) {
    Cache r;
    r.k = c.tensor(k);
    if (!c.ok || r.k->dim() != 4 || !r.k->is_contiguous()) {
        c.ok = false;
        return r;
    }
    const at::IntArrayRef s = r.k->sizes();
    r.v = c.dense(v, r.k->scalar_type(), s);
    r.dtype = dtype_of(*r.k);
    if (r.dtype < 0 || !fits_int(s[0]) || !fits_int(s[1]) || !fits_int(s[2]) || !fits_int(s[3])) c.ok = false;
    if (r.dtype == DSPARK_E4M3) {
        r.k_scale = c.at_dense<uint8_t>(ks, at::kByte, s.slice(0, 3));
        r.v_scale = c.at_dense<uint8_t>(vs, at::kByte, s.slice(0, 3));
    } else if (ks != Py_None || vs != Py_None) {
        c.ok = false;
    }
    r.n_pages = int(s[0]);
    r.heads = int(s[1]);
    r.page_size = int(s[2]);
    r.D = int(s[3]);
    return r;
}

struct Requests {
    int32_t *table = nullptr, *offsets = nullptr, *lens = nullptr;
    int B = 0, max_pages = 0;
};
Requests requests_of(Call &c, PyObject *table, PyObject *offsets, PyObject *lens, int64_t n_rows) {
    Requests r;
    const at::Tensor *t = c.tensor(table);
    if (!c.ok || t->dim() != 2 || t->scalar_type() != at::kInt || !t->is_contiguous() || !fits_int(t->size(1)) ||
        t->size(0) < 1 || t->size(0) > DSPARK_MAX_BATCH || !fits_int(n_rows) || (offsets == Py_None && t->size(0) != n_rows)) {
        c.ok = false;
        return r;
    }
    r.table = static_cast<int32_t *>(t->data_ptr());
    r.B = int(t->size(0));
    r.max_pages = int(t->size(1));
    r.offsets = c.at_dense_or_none<int32_t>(offsets, at::kInt, {r.B + 1});
    r.lens = c.at_dense_or_none<int32_t>(lens, at::kInt, {r.B});
    return r;
}

bool scale_of(PyObject *o, int64_t D, float &s) {
    if (o == Py_None) {
        s = float(1.0 / std::sqrt(double(D)));
        return true;
    }
    if (!PyFloat_Check(o)) return false;
    s = float(PyFloat_AS_DOUBLE(o));
    return true;
}

// workspace: a uint8 tensor of at least `need` bytes
void *workspace_of(Call &c, PyObject *o, size_t need, size_t &bytes) {
    const at::Tensor *t = c.tensor(o);
    if (!c.ok || t->scalar_type() != at::kByte || !t->is_contiguous() || size_t(t->numel()) < need || need == 0) {
        c.ok = false;
        return nullptr;
    }
    bytes = size_t(t->numel());
    return t->data_ptr();
}

// kv_write(k, v, k_cache, v_cache, cache_len, page_table, row_offsets, k_scale, v_scale)
PyObject *kv_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) Py_RETURN_NONE;
    Call c;
    int64_t ks = 0, vs = 0;
    const at::Tensor *k = c.rows(a[0], ks), *v = c.rows(a[1], vs);
    const Cache m = cache_of(c, a[2], a[3], a[7], a[8]);
    if (!c.ok || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type() || k->size(1) != m.heads ||
        k->size(2) != m.D || a[4] == Py_None)
        Py_RETURN_NONE;
    const Requests r = requests_of(c, a[5], a[6], a[4], k->size(0));
    void *s = nullptr;
    const int dt = dtype_of(*k);
    if (dt < 0 || !c.stream(s)) Py_RETURN_NONE;
    return PyLong_FromLong(entry.kv_write(k->data_ptr(), v->data_ptr(), ks, vs, dt, r.offsets, int(k->size(0)), r.lens,
                                          r.table, r.B, r.max_pages, m.heads, m.D, m.k->data_ptr(), m.v->data_ptr(),
                                          m.k_scale, m.v_scale, m.dtype, m.n_pages, m.page_size, s));
}

// kv_read(k_cache, v_cache, page_table, row_offsets, first, k_scale, v_scale, k_out, v_out)
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) Py_RETURN_NONE;
    Call c;
    const Cache m = cache_of(c, a[0], a[1], a[5], a[6]);
    const at::Tensor *ko = c.tensor(a[7]);
    if (!c.ok || ko->dim() != 3 || !ko->is_contiguous() || ko->size(0) == 0 || ko->size(1) != m.heads || ko->size(2) != m.D)
        Py_RETURN_NONE;
    const at::Tensor *vo = c.dense(a[8], ko->scalar_type(), ko->sizes());
    const Requests r = requests_of(c, a[2], a[3], a[4], ko->size(0));
    void *s = nullptr;
    const int dt = dtype_of(*ko);
    if (dt < 0 || !c.stream(s)) Py_RETURN_NONE;
    return PyLong_FromLong(entry.kv_read(m.k->data_ptr(), m.v->data_ptr(), m.k_scale, m.v_scale, m.dtype, m.n_pages,
                                         m.page_size, r.offsets, int(ko->size(0)), r.lens, r.table, r.B, r.max_pages,
                                         m.heads, m.D, ko->data_ptr(), vo->data_ptr(), dt, s));
}

// paged_attention(q, k_cache, v_cache, cache_len, page_table, row_offsets, k_scale, v_scale, scale, causal, max_rows,
//                 out, lse, workspace)
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 14) Py_RETURN_NONE;
    Call c;
    int64_t qs = 0;
    const at::Tensor *q = c.rows(a[0], qs);
    const Cache m = cache_of(c, a[1], a[2], a[6], a[7]);
    float scale = 0.f;
    if (!c.ok || q->size(2) != m.D || a[3] == Py_None || !fits_int(q->size(1)) || !scale_of(a[8], m.D, scale) ||
        !PyBool_Check(a[9]))
        Py_RETURN_NONE;
    const Requests r = requests_of(c, a[4], a[5], a[3], q->size(0));
    if (!c.ok) Py_RETURN_NONE;
    int64_t max_rows = (q->size(0) + r.B - 1) / r.B;
    if (a[10] != Py_None) {
        if (!PyLong_CheckExact(a[10])) Py_RETURN_NONE;
        int overflow = 0;
        max_rows = PyLong_AsLongAndOverflow(a[10], &overflow);
        if (overflow || !fits_int(max_rows)) Py_RETURN_NONE;
    }
    const int heads = int(q->size(1)), dt = dtype_of(*q);
    void *out = c.at_dense(a[11], q->scalar_type(), q->sizes());
    float *lse = c.at_dense_or_none<float>(a[12], at::kFloat, q->sizes().slice(0, 2));
    size_t bytes = 0;
    void *ws = workspace_of(c, a[13], entry.paged_ws(int(max_rows), heads, m.heads, m.D), bytes);
    void *s = nullptr;
    if (dt < 0 || !c.stream(s)) Py_RETURN_NONE;
    return PyLong_FromLong(entry.paged(q->data_ptr(), qs, dt, r.offsets, int(q->size(0)), int(max_rows), r.lens, r.table,
                                       r.B, r.max_pages, heads, m.heads, m.D, m.k->data_ptr(), m.v->data_ptr(), m.k_scale,
                                       m.v_scale, m.dtype, m.n_pages, m.page_size, scale, a[9] == Py_True, out, lse, ws,
                                       bytes, s));
}

// prompt_attention(q, k, v, row_offsets, kv_offsets, scale, causal, out, lse, workspace)
PyObject *prompt_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10) Py_RETURN_NONE;
    Call c;
    int64_t qs = 0, ks = 0, vs = 0;
    const at::Tensor *q = c.rows(a[0], qs), *k = c.rows(a[1], ks), *v = c.rows(a[2], vs);
    const at::Tensor *off = c.tensor(a[3]);
    float scale = 0.f;
    if (!c.ok || k->sizes() != v->sizes() || k->scalar_type() != q->scalar_type() ||
        v->scalar_type() != q->scalar_type() || k->size(2) != q->size(2) || off->dim() != 1 || off->size(0) < 2 ||
        off->size(0) > DSPARK_MAX_BATCH + 1 || off->scalar_type() != at::kInt || !off->is_contiguous() ||
        (a[4] == Py_None && k->size(0) != q->size(0)) || !fits_int(q->size(0)) || !fits_int(k->size(0)) ||
        !fits_int(q->size(1)) || !fits_int(k->size(1)) || !fits_int(q->size(2)) ||
        !scale_of(a[5], q->size(2), scale) || !PyBool_Check(a[6]))
        Py_RETURN_NONE;
    const int B = int(off->size(0)) - 1, rows = int(q->size(0)), keys = int(k->size(0));
    const int heads = int(q->size(1)), kv_heads = int(k->size(1)), D = int(q->size(2)), dt = dtype_of(*q);
    int32_t *kv_off = c.at_dense_or_none<int32_t>(a[4], at::kInt, {B + 1});
    void *out = c.at_dense(a[7], q->scalar_type(), q->sizes());
    float *lse = c.at_dense_or_none<float>(a[8], at::kFloat, q->sizes().slice(0, 2));
    size_t bytes = 0;
    void *ws = workspace_of(c, a[9], entry.prompt_ws(B, rows, keys, heads, kv_heads, D), bytes);
    void *s = nullptr;
    if (dt < 0 || !c.stream(s)) Py_RETURN_NONE;
    return PyLong_FromLong(entry.prompt(q->data_ptr(), k->data_ptr(), v->data_ptr(), qs, ks, vs, dt,
                                        static_cast<int32_t *>(off->data_ptr()), rows, kv_off, keys, B, heads, kv_heads,
                                        D, scale, a[6] == Py_True, out, lse, ws, bytes, s));
}

// bind(addresses of the six entry points, raw_stream, current_device)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "bind: six addresses and two functions");
        return nullptr;
    }
    void *p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
            return nullptr;
        }
    }
    entry.kv_write = reinterpret_cast<decltype(entry.kv_write)>(p[0]);
    entry.kv_read = reinterpret_cast<decltype(entry.kv_read)>(p[1]);
    entry.paged_ws = reinterpret_cast<decltype(entry.paged_ws)>(p[2]);
    entry.paged = reinterpret_cast<decltype(entry.paged)>(p[3]);
    entry.prompt_ws = reinterpret_cast<decltype(entry.prompt_ws)>(p[4]);
    entry.prompt = reinterpret_cast<decltype(entry.prompt)>(p[5]);
    Py_INCREF(a[6]);
    Py_INCREF(a[7]);
    Py_XSETREF(raw_stream, a[6]);
    Py_XSETREF(current_device, a[7]);
    Py_RETURN_NONE;
}

// A C++ exception must not leave a function Python calls: it stands for "not in order".
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

#define METHOD(name) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {METHOD(bind),           METHOD(kv_write), METHOD(kv_read), METHOD(paged_attention),
                         METHOD(prompt_attention), {nullptr, nullptr, 0, nullptr}};
#undef METHOD
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
