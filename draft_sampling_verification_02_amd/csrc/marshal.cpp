// marshal.cpp -- the short way from torch tensors to the cache, rotation,
// attention and logit entry points, for calls whose kernels take a few microseconds.
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
    decltype(&dspark_rotary) rotary;
    decltype(&dspark_kv_append) append;
    decltype(&dspark_window_attention_workspace_size) window_ws;
    decltype(&dspark_window_attention) window;
    decltype(&dspark_logit_rules) rules;
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

// What a rotation takes beside its rows.
struct Turn {
    float *freq = nullptr, eps = 0.f;
    void *q_norm = nullptr, *k_norm = nullptr;
    int rot = 0, norm_dtype = 0;
    bool neighbours = false;
};
Turn turn_of(Call &c, PyObject *freq, PyObject *qn, PyObject *kn, PyObject *eps, PyObject *neighbours, at::ScalarType type,
             int64_t D) {
    Turn t;
    t.norm_dtype = type == at::kHalf ? DSPARK_F16 : DSPARK_BF16;
    if (freq != Py_None) {
        const at::Tensor *f = c.tensor(freq);
        if (!c.ok || f->dim() != 1 || f->scalar_type() != at::kFloat || !f->is_contiguous() || f->size(0) > D) {
            c.ok = false;
            return t;
        }
        t.freq = static_cast<float *>(f->data_ptr());
        t.rot = int(2 * f->size(0));
    }
    PyObject *first = qn != Py_None ? qn : kn;
    if (first != Py_None) {
        const at::Tensor *w = c.tensor(first);
        if (!c.ok) return t;
        const at::ScalarType kind = w->scalar_type() == at::kFloat ? at::kFloat : type;
        if (kind == at::kFloat) t.norm_dtype = DSPARK_F32;
        t.q_norm = c.at_dense_or_none(qn, kind, {D});
        t.k_norm = c.at_dense_or_none(kn, kind, {D});
    }
    if (!PyFloat_Check(eps) || !PyBool_Check(neighbours)) {
        c.ok = false;
        return t;
    }
    t.eps = float(PyFloat_AS_DOUBLE(eps));
    t.neighbours = neighbours == Py_True;
    return t;
}

// rotary(q, k, inv_freq, row_offsets, first, q_norm, k_norm, eps, neighbours, q_out, k_out): q and k both there
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 11) Py_RETURN_NONE;
    Call c;
    int64_t qs = 0, ks = 0, qo = 0, ko = 0;
    const at::Tensor *q = c.rows(a[0], qs), *k = c.rows(a[1], ks), *to_q = c.rows(a[9], qo), *to_k = c.rows(a[10], ko);
    if (!c.ok || q->size(0) != k->size(0) || q->size(2) != k->size(2) || k->scalar_type() != q->scalar_type() ||
        to_q->scalar_type() != q->scalar_type() || to_k->scalar_type() != q->scalar_type() || to_q->sizes() != q->sizes() ||
        to_k->sizes() != k->sizes() || !fits_int(q->size(0)) || !fits_int(q->size(1)) || !fits_int(k->size(1)) ||
        !fits_int(q->size(2)))
        Py_RETURN_NONE;
    int64_t B = q->size(0);
    int32_t *off = nullptr;
    if (a[3] != Py_None) {
        const at::Tensor *t = c.tensor(a[3]);
        if (!c.ok || t->dim() != 1 || t->size(0) < 2) Py_RETURN_NONE;
        B = t->size(0) - 1;
        off = c.at_dense<int32_t>(a[3], at::kInt, {B + 1});
    }
    if (!fits_int(B)) Py_RETURN_NONE;
    int32_t *first = c.at_dense_or_none<int32_t>(a[4], at::kInt, {B});
    const Turn t = turn_of(c, a[2], a[5], a[6], a[7], a[8], q->scalar_type(), q->size(2));
    void *s = nullptr;
    const int dt = dtype_of(*q);
    if (dt < 0 || !c.stream(s)) Py_RETURN_NONE;
    return PyLong_FromLong(entry.rotary(q->data_ptr(), k->data_ptr(), qs, ks, dt, off, int(q->size(0)), first, int(B),
                                        int(q->size(1)), int(k->size(1)), int(q->size(2)), t.freq, t.rot, t.neighbours,
                                        t.q_norm, t.k_norm, t.norm_dtype, t.eps, to_q->data_ptr(), to_k->data_ptr(), qo,
                                        ko, s));
}

// kv_append(q, k, v, inv_freq, k_cache, v_cache, cache_len, page_table, row_offsets, q_norm, k_norm, eps, neighbours,
//           k_scale, v_scale, q_out): q is there
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 16) Py_RETURN_NONE;
    Call c;
    int64_t qs = 0, ks = 0, vs = 0, qo = 0;
    const at::Tensor *q = c.rows(a[0], qs), *k = c.rows(a[1], ks), *v = c.rows(a[2], vs), *to_q = c.rows(a[15], qo);
    const Cache m = cache_of(c, a[4], a[5], a[13], a[14]);
    if (!c.ok || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type() || k->scalar_type() != q->scalar_type() ||
        k->size(1) != m.heads || k->size(2) != m.D || q->size(2) != m.D || q->size(0) != k->size(0) ||
        to_q->sizes() != q->sizes() || to_q->scalar_type() != q->scalar_type() || !fits_int(q->size(1)) || a[6] == Py_None)
        Py_RETURN_NONE;
    const Requests r = requests_of(c, a[7], a[8], a[6], k->size(0));
    const Turn t = turn_of(c, a[3], a[9], a[10], a[11], a[12], k->scalar_type(), m.D);
    void *s = nullptr;
    const int dt = dtype_of(*k);
    if (dt < 0 || !c.stream(s)) Py_RETURN_NONE;
    return PyLong_FromLong(entry.append(q->data_ptr(), k->data_ptr(), v->data_ptr(), qs, ks, vs, dt, r.offsets,
                                        int(k->size(0)), r.lens, r.table, r.B, r.max_pages, int(q->size(1)), m.heads, m.D,
                                        t.freq, t.rot, t.neighbours, t.q_norm, t.k_norm, t.norm_dtype, t.eps,
                                        to_q->data_ptr(), qo, m.k->data_ptr(), m.v->data_ptr(), m.k_scale, m.v_scale,
                                        m.dtype, m.n_pages, m.page_size, s));
}

// a whole number of at least 0 that fits an int
bool count_of(PyObject *o, int &x) {
    if (!PyLong_CheckExact(o)) return false;
    int overflow = 0;
    const long v = PyLong_AsLongAndOverflow(o, &overflow);
    if (overflow || !fits_int(v)) return false;
    x = int(v);
    return true;
}

// window_attention(q, k_cache, v_cache, cache_len, page_table, window, sinks, row_offsets, k_scale, v_scale, scale,
//                  max_rows, out, lse, workspace)
PyObject *window_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 15) Py_RETURN_NONE;
    Call c;
    int64_t qs = 0;
    const at::Tensor *q = c.rows(a[0], qs);
    const Cache m = cache_of(c, a[1], a[2], a[8], a[9]);
    float scale = 0.f;
    int window = 0, sinks = 0;
    if (!c.ok || q->size(2) != m.D || a[3] == Py_None || !fits_int(q->size(1)) || !scale_of(a[10], m.D, scale) ||
        !count_of(a[5], window) || !count_of(a[6], sinks))
        Py_RETURN_NONE;
    const Requests r = requests_of(c, a[4], a[7], a[3], q->size(0));
    if (!c.ok) Py_RETURN_NONE;
    int max_rows = int((q->size(0) + r.B - 1) / r.B);
    if (a[11] != Py_None && !count_of(a[11], max_rows)) Py_RETURN_NONE;
    const int heads = int(q->size(1)), dt = dtype_of(*q);
    void *out = c.at_dense(a[12], q->scalar_type(), q->sizes());
    float *lse = c.at_dense_or_none<float>(a[13], at::kFloat, q->sizes().slice(0, 2));
    size_t bytes = 0;
    void *ws = workspace_of(c, a[14], entry.window_ws(max_rows, heads, m.heads, m.D), bytes);
    void *s = nullptr;
    if (dt < 0 || !c.stream(s)) Py_RETURN_NONE;
    return PyLong_FromLong(entry.window(q->data_ptr(), qs, dt, r.offsets, int(q->size(0)), max_rows, r.lens, r.table, r.B,
                                        r.max_pages, heads, m.heads, m.D, m.k->data_ptr(), m.v->data_ptr(), m.k_scale,
                                        m.v_scale, m.dtype, m.n_pages, m.page_size, window, sinks, scale, out, lse, ws,
                                        bytes, s));
}

// logit_rules(logits, row_offsets, history, history_len, prompt_len, drafts, repetition, frequency, presence,
//             bias_offsets, bias_ids, bias_values, masks, mask_index, out)
PyObject *logit_rules(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 15) Py_RETURN_NONE;
    Call c;
    auto padded = [&](PyObject *o, int64_t &stride) -> const at::Tensor * {
        const at::Tensor *t = c.tensor(o);
        if (!c.ok || t->dim() != 2 || t->size(0) == 0 || t->size(1) == 0 || t->stride(1) != 1) {
            c.ok = false;
            return nullptr;
        }
        stride = t->size(0) > 1 ? t->stride(0) : t->size(1);
        return t;
    };
    int64_t stride = 0, out_stride = 0;
    const at::Tensor *x = padded(a[0], stride), *out = padded(a[14], out_stride);
    if (!c.ok || out->scalar_type() != at::kFloat || out->sizes() != x->sizes() || !fits_int(x->size(0)) ||
        !fits_int(x->size(1)))
        Py_RETURN_NONE;
    const int dt = x->scalar_type() == at::kFloat ? DSPARK_F32 : dtype_of(*x);
    if (dt < 0 || dt == DSPARK_E4M3) Py_RETURN_NONE;
    const int64_t rows = x->size(0), V = x->size(1);
    int64_t B = rows;
    int32_t *off = nullptr;
    if (a[1] != Py_None) {
        const at::Tensor *t = c.tensor(a[1]);
        if (!c.ok || t->dim() != 1 || t->size(0) < 2) Py_RETURN_NONE;
        B = t->size(0) - 1;
        off = c.at_dense<int32_t>(a[1], at::kInt, {B + 1});
    }
    if (!fits_int(B)) Py_RETURN_NONE;
    auto table = [&](PyObject *o, int64_t lines, int64_t &width) -> int32_t * {
        if (o == Py_None) return nullptr;
        const at::Tensor *t = c.tensor(o);
        if (!c.ok || t->dim() != 2 || !fits_int(t->size(1)) || (lines >= 0 && t->size(0) != lines) || !fits_int(t->size(0)) ||
            t->scalar_type() != at::kInt || !t->is_contiguous()) {
            c.ok = false;
            return nullptr;
        }
        width = t->size(1);
        return static_cast<int32_t *>(t->data_ptr());
    };
    int64_t width = 0, gamma = 0, words = 0, n_masks = 0, n_biases = 0;
    int32_t *history = table(a[2], B, width), *drafts = table(a[5], B, gamma), *masks = table(a[12], -1, words);
    int32_t *history_len = c.at_dense_or_none<int32_t>(a[3], at::kInt, {B});
    int32_t *prompt_len = c.at_dense_or_none<int32_t>(a[4], at::kInt, {B});
    float *rep = c.at_dense_or_none<float>(a[6], at::kFloat, {B}), *freq = c.at_dense_or_none<float>(a[7], at::kFloat, {B});
    float *pres = c.at_dense_or_none<float>(a[8], at::kFloat, {B});
    int32_t *bias_off = c.at_dense_or_none<int32_t>(a[9], at::kInt, {B + 1}), *ids = nullptr;
    float *values = nullptr;
    if (bias_off) {
        const at::Tensor *t = c.tensor(a[10]);
        if (!c.ok || !fits_int(t->numel())) Py_RETURN_NONE;
        n_biases = t->numel();
        ids = c.at_dense<int32_t>(a[10], at::kInt, {n_biases});
        values = c.at_dense<float>(a[11], at::kFloat, {n_biases});
    }
    int32_t *index = c.at_dense_or_none<int32_t>(a[13], at::kInt, {rows});
    // (an empty tensor has no address: what is there is told by the argument)
    const bool masked = a[12] != Py_None;
    if (!c.ok || (a[2] != Py_None && !history_len) || (masked && (!index || words < (V + 31) / 32))) Py_RETURN_NONE;
    if (masked) n_masks = THPVariable_Unpack(a[12]).size(0);
    void *s = nullptr;
    if (!c.stream(s)) Py_RETURN_NONE;
    return PyLong_FromLong(entry.rules(x->data_ptr(), stride, dt, off, int(rows), int(B), int(V), history, int(width),
                                       history_len, prompt_len, drafts, int(gamma), rep, freq, pres, bias_off, ids, values,
                                       int(n_biases), masks, int(n_masks), words, index,
                                       static_cast<float *>(out->data_ptr()), out_stride, s));
}

// bind(addresses of the eleven entry points, raw_stream, current_device)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13) {
        PyErr_SetString(PyExc_TypeError, "bind: eleven addresses and two functions");
        return nullptr;
    }
    void *p[11];
    for (int i = 0; i < 11; ++i) {
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
    entry.rotary = reinterpret_cast<decltype(entry.rotary)>(p[6]);
    entry.append = reinterpret_cast<decltype(entry.append)>(p[7]);
    entry.window_ws = reinterpret_cast<decltype(entry.window_ws)>(p[8]);
    entry.window = reinterpret_cast<decltype(entry.window)>(p[9]);
    entry.rules = reinterpret_cast<decltype(entry.rules)>(p[10]);
    Py_INCREF(a[11]);
    Py_INCREF(a[12]);
    Py_XSETREF(raw_stream, a[11]);
    Py_XSETREF(current_device, a[12]);
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
                         METHOD(prompt_attention), METHOD(rotary), METHOD(kv_append), METHOD(window_attention),
                         METHOD(logit_rules), {nullptr, nullptr, 0, nullptr}};
#undef METHOD
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
