/* The marshalling of the operators over caller-held caches, as a CPython module: it
 * reads the tensors' shapes, strides, types and addresses, checks that they belong together
 * (ValueError) and calls the library.  Their smallest calls take the GPU 2 to 7 us, and the same
 * checks in Python with a ctypes call took the host 6 to 8 us.
 *
 * The library's functions and torch's objects are handed over once (setup), so the module
 * links to neither.  Functions return the library's status. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "qd.h"

typedef qd_status (*rows_fn)(const qd_kv_cache *, const void *, const void *, int, int, int64_t, int64_t, int64_t,
                             const int32_t *, const int32_t *, void *);
typedef qd_status (*attn_fn)(const qd_kv_cache *, const qd_kv_cache *, int, const void *, int64_t, int64_t, void *,
                             int64_t, int64_t, int, int, int, float, const int32_t *, const int32_t *, int, void *,
                             size_t, void *);
typedef qd_status (*space_fn)(const qd_kv_cache *, const qd_kv_cache *, int, int, int, int, int, size_t *);
typedef qd_status (*verify_fn)(const float *, int64_t, int64_t, const float *, int64_t, int64_t, const int32_t *,
                               const int32_t *, const float *, int, int, int, int32_t *, int32_t *, void *);
typedef qd_status (*paged_fn)(const qd_kv_cache *, const int32_t *, int64_t, int, int, const void *, int64_t, int64_t, void *, int64_t,
                              int64_t, int, int, int, float, const int32_t *, const int32_t *, int, void *, size_t, void *);
typedef qd_status (*paged_space_fn)(const qd_kv_cache *, int, int, int, int, int, int, size_t *);
typedef qd_status (*prompt_fn)(const void *, int64_t, const void *, int64_t, const void *, int64_t, void *, int64_t, int, int, int, int, int,
                               float, const int32_t *, const int32_t *, int, void *, size_t, void *);
typedef qd_status (*prompt_space_fn)(int, int, int, int, int, int, size_t *);
typedef qd_status (*rope_fn)(const qd_rope_rows *, void *);

static rows_fn f_append, f_read;
static attn_fn f_attn;
static space_fn f_space;
static verify_fn f_verify;
static rope_fn f_rope;
static paged_fn f_paged;
static paged_space_fn f_paged_space;
static prompt_fn f_prompt;
static prompt_space_fn f_prompt_space;
static PyObject *t_f32, *t_bf16, *t_i32;               /* torch's types */
static PyObject *raw_stream, *capturing;               /* its current raw stream of a device; whether that is being captured */
static PyObject *s_shape, *s_stride, *s_dtype, *s_ptr, *s_device, *s_stream;

/* Scratch of torch's current streams, one tensor per device and stream, held here.  Calls on one stream follow one another, and the interpreter's lock is held from the look-up to the last launch, so two host threads cannot
 * interleave theirs. */
static struct {
    long dev;
    void *stream, *ptr;
    size_t size;
    PyObject *tensor;
} scratch[64];
static int n_scratch;

typedef struct {
    int nd;
    int64_t shape[4], stride[4];
    PyObject *type;                     /* compared, not owned: the types are torch's own */
    void *ptr;
} Tensor;

static int bad(const char *what) {
    PyErr_SetString(PyExc_ValueError, what);
    return 0;
}

static int int_items(PyObject *t, int64_t *to, int *n) {
    if (!t) return 0;
    const int ok = PyTuple_Check(t) && PyTuple_GET_SIZE(t) <= 4;
    if (ok) {
        *n = (int)PyTuple_GET_SIZE(t);
        for (int i = 0; i < *n; ++i) to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    }
    Py_DECREF(t);
    return PyErr_Occurred() ? 0 : ok ? 1 : bad("a tensor of at most four axes is wanted");
}

static int read_tensor(PyObject *t, Tensor *o) {
    int ns = 0;
    if (!int_items(PyObject_GetAttr(t, s_shape), o->shape, &o->nd)) return 0;
    if (!int_items(PyObject_CallMethodNoArgs(t, s_stride), o->stride, &ns)) return 0;
    if (ns != o->nd) return bad("a strided tensor is wanted");
    PyObject *type = PyObject_GetAttr(t, s_dtype);
    if (!type) return 0;
    o->type = type;
    Py_DECREF(type);
    PyObject *p = PyObject_CallMethodNoArgs(t, s_ptr);
    if (!p) return 0;
    o->ptr = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return !PyErr_Occurred();
}

/* n contiguous int32 values (any number, where n is below 0: *found then), or None */
static int read_some_ints(PyObject *t, int64_t n, int64_t *found, const int32_t **to, const char *what) {
    *to = NULL;
    if (t == Py_None) return 1;
    Tensor x;
    if (!read_tensor(t, &x)) return 0;
    int64_t count = 1;
    int ok = x.type == t_i32;
    for (int i = x.nd - 1; i >= 0; --i) {
        if (x.shape[i] != 1 && x.stride[i] != count) ok = 0;
        count *= x.shape[i];
    }
    if (n < 0 && x.nd == 1) n = *found = count;
    if (!ok || count != n) {
        if (n < 0)
            PyErr_Format(PyExc_ValueError, "%s must be one axis of contiguous int32 values", what);
        else
            PyErr_Format(PyExc_ValueError, "%s must be %lld contiguous int32 values", what, (long long)n);
        return 0;
    }
    *to = (const int32_t *)x.ptr;
    return 1;
}
static int read_ints(PyObject *t, int64_t n, const int32_t **to, const char *what) { return read_some_ints(t, n, NULL, to, what); }

static int type_of(const Tensor *t, int *dtype) {
    if (t->type == t_bf16)
        *dtype = QD_BF16;
    else if (t->type == t_f32)
        *dtype = QD_F32;
    else
        return bad("fp32 or bf16 wanted");
    return 1;
}

/* stream: a torch.cuda.Stream, or None for the current one of t's device (*device then, else -1) */
static int stream_of(PyObject *stream, PyObject *t, void **to, long *device) {
    PyObject *v;
    *device = -1;
    if (stream != Py_None) {
        v = PyObject_GetAttr(stream, s_stream);
    } else {
        PyObject *dev = PyObject_CallMethodNoArgs(t, s_device);
        if (!dev) return 0;
        *device = PyLong_AsLong(dev);
        if (*device < 0) {              /* host memory, which the call will refuse */
            Py_DECREF(dev);
            *to = NULL;
            return !PyErr_Occurred();
        }
        v = PyObject_CallOneArg(raw_stream, dev);
        Py_DECREF(dev);
    }
    if (!v) return 0;
    *to = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

static int same_layout(const Tensor *a, const Tensor *b) {
    if (a->nd != b->nd || a->type != b->type) return 0;
    for (int i = 0; i < a->nd; ++i)
        if (a->shape[i] != b->shape[i] || a->stride[i] != b->stride[i]) return 0;
    return 1;
}

/* sizes that the library takes as int */
static int fits(const Tensor *t) {
    for (int i = 0; i < t->nd; ++i)
        if (t->shape[i] > INT32_MAX) return bad("an axis is too long");
    return 1;
}

#define NARGS(n)                                                    \
    if (nargs != (n)) {                                             \
        PyErr_SetString(PyExc_TypeError, #n " arguments wanted");   \
        return NULL;                                                \
    }

/* rows(read, cache, k_rows, v_rows, lengths, n_new, stream) */
static PyObject *py_rows(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    NARGS(7)
    const qd_kv_cache *c = (const qd_kv_cache *)PyLong_AsVoidPtr(a[1]);
    Tensor k, v;
    const int32_t *lengths, *n_new;
    void *s;
    long dev;
    int dtype;
    if (PyErr_Occurred() || !read_tensor(a[2], &k) || !read_tensor(a[3], &v)) return NULL;
    if (k.nd != 4 || !same_layout(&k, &v) || k.shape[0] != c->n_streams || k.shape[2] != c->n_kv_heads ||
        k.shape[3] != c->head_dim || k.stride[3] != 1) {
        PyErr_Format(PyExc_ValueError, "k_rows and v_rows must be alike: [%d, tokens, %d, %d], heads contiguous",
                     c->n_streams, c->n_kv_heads, c->head_dim);
        return NULL;
    }
    if (!fits(&k) || !type_of(&k, &dtype) || !read_ints(a[4], c->n_streams, &lengths, "lengths") ||
        !read_ints(a[5], c->n_streams, &n_new, "n_new") || !stream_of(a[6], a[2], &s, &dev))
        return NULL;
    const qd_status st = (a[0] == Py_True ? f_read : f_append)(
        c, k.ptr, v.ptr, dtype, (int)k.shape[1], k.shape[0] > 1 ? k.stride[0] : 0, k.shape[1] > 1 ? k.stride[1] : 0,
        k.shape[2] > 1 ? k.stride[2] : 0, lengths, n_new, s);
    return PyLong_FromLong(st);
}

static int opt_int(PyObject *o, int otherwise, int *to) {
    *to = otherwise;
    if (o == Py_None) return 1;
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return 0;
    if (v > INT32_MAX || v < INT32_MIN) return bad("a number is too large");
    *to = (int)v;
    return 1;
}

/* The scratch kept for a stream, where it has `need` bytes and the stream is not being captured (the replays may run beside anything):
 * *ws NULL otherwise */
static int find_scratch(long dev, void *stream, size_t need, void **ws, size_t *have) {
    *ws = NULL, *have = 0;
    if (dev < 0) return 1;
    PyObject *cap = PyObject_CallNoArgs(capturing);
    if (!cap) return 0;
    const int is = PyObject_IsTrue(cap);
    Py_DECREF(cap);
    for (int i = 0; !is && i < n_scratch; ++i)
        if (scratch[i].dev == dev && scratch[i].stream == stream && scratch[i].size >= need) {
            *ws = scratch[i].ptr, *have = scratch[i].size;
            break;
        }
    return 1;
}

/* q and out: [streams, tokens, q_heads, head_dim] of one type, heads contiguous; B < 0: any number of streams */
static int read_queries(PyObject *qo, PyObject *oo, int64_t B, int64_t D, Tensor *q, Tensor *o, int *dtype) {
    if (!read_tensor(qo, q) || !read_tensor(oo, o)) return 0;
    if (B < 0) B = q->nd == 4 ? q->shape[0] : 0;
    if (q->nd != 4 || o->nd != 4 || q->type != o->type || q->shape[0] != B || q->shape[3] != D || o->shape[0] != B ||
        o->shape[1] != q->shape[1] || o->shape[2] != q->shape[2] || o->shape[3] != D) {
        PyErr_Format(PyExc_ValueError, "q and out must be [%lld, tokens, q_heads, %lld] of one type", (long long)B, (long long)D);
        return 0;
    }
    if (q->stride[3] != 1 || o->stride[3] != 1 || (q->shape[2] > 1 && (q->stride[2] != D || o->stride[2] != D)))
        return bad("the heads of q and out must be contiguous");
    return fits(q) && type_of(q, dtype);
}

static int read_scale(PyObject *o, int64_t d, float *to) {
    double scale = 1.0 / (d == 64 ? 8.0 : 11.313708498984761);   /* head_dim ** -0.5 */
    if (o != Py_None) {
        scale = PyFloat_AsDouble(o);
        if (scale == -1.0 && PyErr_Occurred()) return 0;
    }
    *to = (float)scale;
    return 1;
}

/* attn(q, cache, lengths, out, n_new, max_length, scale, prefix, prefix_length, workspace, workspace_bytes, stream):
 * the status; with workspace None and no scratch kept for the stream that is large enough (in a capture: none is used, the
 * replays may run beside anything), the bytes that the call needs instead of making it */
static PyObject *py_attn(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    NARGS(12)
    const qd_kv_cache *c = (const qd_kv_cache *)PyLong_AsVoidPtr(a[1]);
    const qd_kv_cache *p = a[7] == Py_None ? NULL : (const qd_kv_cache *)PyLong_AsVoidPtr(a[7]);
    Tensor q, o;
    const int32_t *lengths, *n_new;
    void *s, *ws = NULL;
    long dev;
    int dtype, most, plen;
    size_t have = 0;
    const int64_t D = c->head_dim, B = c->n_streams;
    if (PyErr_Occurred() || !read_queries(a[0], a[3], B, D, &q, &o, &dtype)) return NULL;
    if (!opt_int(a[5], c->smax, &most) || !opt_int(a[8], p ? p->smax : 0, &plen))
        return NULL;
    if (p && p->n_streams != 1) {
        bad("the prefix is a cache of one stream");
        return NULL;
    }
    if (!p && plen) {
        bad("prefix_length without a prefix");
        return NULL;
    }
    if (plen == 0) p = NULL;
    float scale;
    if (!read_scale(a[6], D, &scale) || !read_ints(a[2], B, &lengths, "lengths") || !read_ints(a[4], B, &n_new, "n_new") || !stream_of(a[11], a[0], &s, &dev))
        return NULL;
    const int T = (int)q.shape[1], QH = (int)q.shape[2];
    if (a[9] != Py_None) {
        ws = PyLong_AsVoidPtr(a[9]);
        have = PyLong_AsSize_t(a[10]);
        if (PyErr_Occurred()) return NULL;
    } else {
        size_t need = 0;
        const qd_status st = f_space(c, p, plen, dtype, T, QH, most, &need);
        if (st != QD_OK) return PyLong_FromLong(st);
        if (need) {
            if (!find_scratch(dev, s, need, &ws, &have)) return NULL;
            if (!ws) return PyLong_FromSize_t(need);
        }
    }
    return PyLong_FromLong(f_attn(c, p, plen, q.ptr, B > 1 ? q.stride[0] : 0, T > 1 ? q.stride[1] : 0, o.ptr,
                                  B > 1 ? o.stride[0] : 0, T > 1 ? o.stride[1] : 0, dtype, T, QH, scale, lengths,
                                  n_new, most, ws, have, s));
}

/* page_table: int32 [streams, pages of one], a stream's contiguous */
static int read_table(PyObject *o, int64_t streams, const int32_t **to, int64_t *stride, int *pages) {
    Tensor t;
    if (!read_tensor(o, &t)) return 0;
    if (t.type != t_i32 || t.nd != 2 || t.shape[0] != streams || (t.shape[1] > 1 && t.stride[1] != 1)) {
        PyErr_Format(PyExc_ValueError, "page_table must be int32 [%lld, pages], rows contiguous", (long long)streams);
        return 0;
    }
    *to = (const int32_t *)t.ptr, *stride = t.shape[0] > 1 ? t.stride[0] : 0, *pages = (int)t.shape[1];
    return fits(&t);
}

/* paged(q, pages, page_table, lengths, out, n_new, max_length, scale, workspace, workspace_bytes, stream): as attn */
static PyObject *py_paged(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    NARGS(11)
    const qd_kv_cache *c = (const qd_kv_cache *)PyLong_AsVoidPtr(a[1]);
    Tensor q, o;
    const int32_t *lengths, *n_new, *table;
    void *s, *ws = NULL;
    long dev;
    int dtype, most, per;
    int64_t table_stride;
    size_t have = 0;
    float scale;
    if (PyErr_Occurred()) return NULL;
    const int64_t D = c->head_dim;
    if (!read_queries(a[0], a[4], -1, D, &q, &o, &dtype)) return NULL;
    const int64_t B = q.shape[0];
    if (!read_table(a[2], B, &table, &table_stride, &per)) return NULL;
    const int64_t named = (int64_t)per * c->smax;
    if (!opt_int(a[6], named > INT32_MAX ? INT32_MAX : (int)named, &most) || !read_scale(a[7], D, &scale) ||
        !read_ints(a[3], B, &lengths, "lengths") || !read_ints(a[5], B, &n_new, "n_new") || !stream_of(a[10], a[0], &s, &dev))
        return NULL;
    const int T = (int)q.shape[1], QH = (int)q.shape[2];
    if (a[8] != Py_None) {
        ws = PyLong_AsVoidPtr(a[8]);
        have = PyLong_AsSize_t(a[9]);
        if (PyErr_Occurred()) return NULL;
    } else {
        size_t need = 0;
        const qd_status st = f_paged_space(c, (int)B, per, dtype, T, QH, most, &need);
        if (st != QD_OK) return PyLong_FromLong(st);
        if (need) {
            if (!find_scratch(dev, s, need, &ws, &have)) return NULL;
            if (!ws) return PyLong_FromSize_t(need);
        }
    }
    return PyLong_FromLong(f_paged(c, table, table_stride, per, (int)B, q.ptr, B > 1 ? q.stride[0] : 0, T > 1 ? q.stride[1] : 0, o.ptr,
                                   B > 1 ? o.stride[0] : 0, T > 1 ? o.stride[1] : 0, dtype, T, QH, scale, lengths, n_new, most, ws, have,
                                   s));
}

/* verify(target_probs, draft_ids, u, out_ids, n_accepted, draft_probs, n_draft, stream) */
static PyObject *py_verify(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    NARGS(8)
    Tensor p, d, u, q;
    const int32_t *ids, *out, *acc, *n_draft;
    void *s;
    long dev;
    if (!read_tensor(a[0], &p) || !read_tensor(a[1], &d) || !read_tensor(a[2], &u)) return NULL;
    if (d.nd != 2) {
        bad("draft_ids must be [streams, tokens]");
        return NULL;
    }
    const int64_t B = d.shape[0], T = d.shape[1];
    if (p.nd != 3 || p.type != t_f32 || p.shape[0] != B || p.shape[1] != T + 1 || p.stride[2] != 1) {
        PyErr_Format(PyExc_ValueError, "target_probs must be fp32 [%lld, %lld, vocab], rows contiguous", (long long)B,
                     (long long)T + 1);
        return NULL;
    }
    const int64_t V = p.shape[2];
    memset(&q, 0, sizeof q);
    if (a[5] != Py_None) {
        if (!read_tensor(a[5], &q)) return NULL;
        if (q.nd != 3 || q.type != t_f32 || q.shape[0] != B || q.shape[1] != T || q.shape[2] != V || q.stride[2] != 1) {
            PyErr_Format(PyExc_ValueError, "draft_probs must be fp32 [%lld, %lld, %lld], rows contiguous", (long long)B,
                         (long long)T, (long long)V);
            return NULL;
        }
    }
    if (u.nd != 2 || u.type != t_f32 || u.shape[0] != B || u.shape[1] != T + 1 || u.stride[1] != 1 ||
        (B > 1 && u.stride[0] != T + 1)) {
        PyErr_Format(PyExc_ValueError, "u must be contiguous fp32 [%lld, %lld]", (long long)B, (long long)T + 1);
        return NULL;
    }
    if (!fits(&p) || !read_ints(a[1], B * T, &ids, "draft_ids") || !read_ints(a[3], B * (T + 1), &out, "out_ids") ||
        !read_ints(a[4], B, &acc, "n_accepted") || !read_ints(a[6], B, &n_draft, "n_draft") || !stream_of(a[7], a[0], &s, &dev))
        return NULL;
    return PyLong_FromLong(f_verify((const float *)p.ptr, B > 1 ? p.stride[0] : 0, p.stride[1], (const float *)q.ptr,
                                    B > 1 ? q.stride[0] : 0, T > 1 ? q.stride[1] : 0, ids, n_draft, (const float *)u.ptr,
                                    (int)B, (int)T, (int)V, (int32_t *)out, (int32_t *)acc, s));
}

/* A tensor [tokens, heads, head_dim] whose heads are contiguous; tokens < 0: any.  None: a null pointer. */
static int read_heads(PyObject *o, const char *what, int64_t tokens, int64_t heads, int64_t d, Tensor *t) {
    memset(t, 0, sizeof *t);
    if (o == Py_None) return 1;
    if (!read_tensor(o, t)) return 0;
    if (t->nd != 3 || (tokens >= 0 && t->shape[0] != tokens) || (heads >= 0 && t->shape[1] != heads) || (d >= 0 && t->shape[2] != d) ||
        (t->shape[2] > 1 && t->stride[2] != 1) || (t->shape[1] > 1 && t->stride[1] != t->shape[2])) {
        PyErr_Format(PyExc_ValueError, "%s must be [tokens, heads, head_dim], a token's heads contiguous", what);
        return 0;
    }
    return fits(t);
}
static int64_t token_stride(const Tensor *t) { return t->shape[0] > 1 ? t->stride[0] : t->shape[1] * t->shape[2]; }

/* contiguous fp32 values of n columns: a vector (rows NULL) or rows of them; None: a null pointer */
static int read_floats(PyObject *o, const char *what, int64_t n, int64_t *rows, const float **to) {
    Tensor t;
    *to = NULL;
    if (o == Py_None) return 1;
    if (!read_tensor(o, &t)) return 0;
    if (t.type != t_f32 || t.nd != (rows ? 2 : 1) || t.shape[t.nd - 1] != n || t.stride[t.nd - 1] != 1 ||
        (rows && t.shape[0] > 1 && t.stride[0] != n)) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous fp32 of %lld columns", what, (long long)n);
        return 0;
    }
    if (rows) *rows = t.shape[0];
    *to = (const float *)t.ptr;
    return fits(&t);
}

/* rope(q, k, v, q_out, k_out, v_out, cos, sin, lengths, offsets, n_new, positions, mrope_h, q_gamma, k_gamma, eps, pages, page_table,
 * stream) */
static PyObject *py_rope(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    NARGS(19)
    Tensor q, k, v, qo, ko, vo;
    qd_rope_rows r;
    memset(&r, 0, sizeof r);
    if (a[0] == Py_None || a[1] == Py_None || a[3] == Py_None) {
        bad("q, k and q_out are wanted");
        return NULL;
    }
    if (!read_heads(a[0], "q", -1, -1, -1, &q)) return NULL;
    const int64_t N = q.shape[0], D = q.shape[2];
    if (!read_heads(a[1], "k", N, -1, D, &k)) return NULL;
    const int64_t H = k.shape[1];
    if (!read_heads(a[2], "v", N, H, D, &v) || !read_heads(a[3], "q_out", N, q.shape[1], D, &qo) ||
        !read_heads(a[4], "k_out", N, H, D, &ko) || !read_heads(a[5], "v_out", N, H, D, &vo))
        return NULL;
    if (k.type != q.type || (v.ptr && v.type != q.type) || (ko.ptr && ko.type != qo.type) || (vo.ptr && vo.type != qo.type)) {
        bad("q, k, v are of one type, and their results of one");
        return NULL;
    }
    if (!type_of(&q, &r.dtype) || !type_of(&qo, &r.out_dtype)) return NULL;
    int64_t n_cos = 0, n_sin = 0;
    if (!read_floats(a[6], "cos", D / 2, &n_cos, &r.cos) || !read_floats(a[7], "sin", D / 2, &n_sin, &r.sin) ||
        !read_floats(a[13], "q_gamma", D, NULL, &r.q_gamma) || !read_floats(a[14], "k_gamma", D, NULL, &r.k_gamma))
        return NULL;
    if (n_cos != n_sin) {
        bad("cos and sin have the same rows");
        return NULL;
    }
    int64_t B = 0;
    if (!read_some_ints(a[8], -1, &B, &r.lengths, "lengths") || !read_ints(a[9], B + 1, &r.offsets, "offsets") ||
        !read_ints(a[10], B, &r.n_new, "n_new") || !opt_int(a[12], 0, &r.mrope_h) ||
        !read_ints(a[11], r.mrope_h ? 3 * N : N, &r.positions, "positions"))
        return NULL;
    r.eps = PyFloat_AsDouble(a[15]);
    if (r.eps == -1.0 && PyErr_Occurred()) return NULL;
    if ((a[16] == Py_None) != (a[17] == Py_None)) {
        bad("pages and page_table come together");
        return NULL;
    }
    if (a[16] != Py_None) {
        r.pages = (const qd_kv_cache *)PyLong_AsVoidPtr(a[16]);
        if (PyErr_Occurred() || !read_table(a[17], B, &r.page_table, &r.table_stride, &r.table_pages)) return NULL;
    }
    void *s;
    long dev;
    if (!stream_of(a[18], a[0], &s, &dev)) return NULL;
    if (N == 0) return PyLong_FromLong(QD_OK);
    r.q = q.ptr, r.k = k.ptr, r.v = v.ptr, r.q_out = qo.ptr, r.k_out = ko.ptr, r.v_out = vo.ptr;
    r.q_stride = token_stride(&q), r.k_stride = token_stride(&k), r.v_stride = v.ptr ? token_stride(&v) : 0;
    r.q_out_stride = token_stride(&qo), r.k_out_stride = ko.ptr ? token_stride(&ko) : 0, r.v_out_stride = vo.ptr ? token_stride(&vo) : 0;
    r.n_tokens = (int)N, r.n_q_heads = (int)q.shape[1], r.n_kv_heads = (int)H, r.head_dim = (int)D;
    r.rope_rows = (int)n_cos, r.n_streams = (int)B;
    return PyLong_FromLong(f_rope(&r, s));
}

/* prompt(q, k, v, out, offsets, kv_offsets, scale, workspace, workspace_bytes, stream): as attn */
static PyObject *py_prompt(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    NARGS(10)
    Tensor q, k, v, o;
    const int32_t *offsets, *kv_offsets;
    void *s, *ws = NULL;
    long dev;
    size_t have = 0;
    float scale;
    for (int i = 0; i < 5; ++i)
        if (a[i] == Py_None) {
            bad("q, k, v, out and offsets are wanted");
            return NULL;
        }
    if (!read_heads(a[0], "q", -1, -1, -1, &q)) return NULL;
    const int64_t N = q.shape[0], QH = q.shape[1], D = q.shape[2];
    if (!read_heads(a[1], "k", -1, -1, D, &k)) return NULL;
    const int64_t M = k.shape[0], H = k.shape[1];
    if (!read_heads(a[2], "v", M, H, D, &v) || !read_heads(a[3], "out", N, QH, D, &o)) return NULL;
    if (q.type != t_bf16 || k.type != t_bf16 || v.type != t_bf16 || o.type != t_bf16) {
        bad("q, k, v and out must be bf16");
        return NULL;
    }
    int64_t B = 0;
    if (!read_some_ints(a[4], -1, &B, &offsets, "offsets")) return NULL;
    if (--B < 0) {
        bad("offsets must be [sequences + 1]");
        return NULL;
    }
    if ( !read_ints(a[5], B + 1, &kv_offsets, "kv_offsets") || !read_scale(a[6], D, &scale) ||
        !stream_of(a[9], a[0], &s, &dev))
        return NULL;
    if (!kv_offsets && M != N) {
        bad("k has other rows than q: kv_offsets are wanted");
        return NULL;
    }
    if (B > INT32_MAX) {
        bad("too many sequences");
        return NULL;
    }
    if (N == 0 || B == 0) return PyLong_FromLong(QD_OK);
    if (a[7] != Py_None) {
        ws = PyLong_AsVoidPtr(a[7]);
        have = PyLong_AsSize_t(a[8]);
        if (PyErr_Occurred()) return NULL;
    } else {
        size_t need = 0;
        const qd_status st = f_prompt_space((int)N, (int)M, (int)B, (int)QH, (int)H, (int)D, &need);
        if (st != QD_OK) return PyLong_FromLong(st);
        if (need) {
            if (!find_scratch(dev, s, need, &ws, &have)) return NULL;
            if (!ws) return PyLong_FromSize_t(need);
        }
    }
    return PyLong_FromLong(f_prompt(q.ptr, token_stride(&q), k.ptr, token_stride(&k), v.ptr, token_stride(&v), o.ptr, token_stride(&o), (int)N,
                                    (int)M, (int)QH, (int)H, (int)D, scale, offsets, kv_offsets, (int)B, ws, have, s));
}

/* keep(device, stream, tensor, pointer, bytes): scratch of a stream from now on, where there is room to note it.  Address
 * and tensor change together, so another thread's call between the two cannot leave an address of freed memory. */
static PyObject *py_keep(PyObject *self, PyObject *args) {
    long dev;
    unsigned long long stream, ptr, size;
    PyObject *tensor, *before = NULL;
    if (!PyArg_ParseTuple(args, "lKOKK", &dev, &stream, &tensor, &ptr, &size)) return NULL;
    int i = 0;
    while (i < n_scratch && (scratch[i].dev != dev || scratch[i].stream != (void *)(uintptr_t)stream)) ++i;
    if (i == 64) Py_RETURN_FALSE;
    scratch[i].dev = dev, scratch[i].stream = (void *)(uintptr_t)stream;
    scratch[i].ptr = (void *)(uintptr_t)ptr, scratch[i].size = (size_t)size;
    if (i == n_scratch)
        ++n_scratch;
    else
        before = scratch[i].tensor;
    Py_INCREF(tensor);
    scratch[i].tensor = tensor;
    Py_XDECREF(before);                 /* to the stream's allocator, which hands it to later work of the stream only */
    Py_RETURN_TRUE;
}

/* release(): gives up the scratch of all streams.  What still runs on one keeps its memory to itself: the allocator hands it to
 * later work of that stream only. */
static PyObject *py_release(PyObject *self, PyObject *none) {
    PyObject *held[64];
    const int n = n_scratch;
    for (int i = 0; i < n; ++i) held[i] = scratch[i].tensor;
    n_scratch = 0;                      /* first: what a tensor's end sets off finds none */
    for (int i = 0; i < n; ++i) Py_DECREF(held[i]);
    Py_RETURN_NONE;
}

/* setup(append, read, attn, workspace, verify, rope, paged, its workspace, prompt, its workspace: addresses; float32, bfloat16, int32, current raw stream, whether it is being
 * captured: torch's) */
static PyObject *py_setup(PyObject *self, PyObject *args) {
    unsigned long long f[10];
    if (!PyArg_ParseTuple(args, "KKKKKKKKKKOOOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8],
                          &f[9], &t_f32, &t_bf16, &t_i32, &raw_stream,
                          &capturing))
        return NULL;
    Py_INCREF(t_f32), Py_INCREF(t_bf16), Py_INCREF(t_i32), Py_INCREF(raw_stream), Py_INCREF(capturing);
    f_append = (rows_fn)(uintptr_t)f[0], f_read = (rows_fn)(uintptr_t)f[1], f_attn = (attn_fn)(uintptr_t)f[2];
    f_space = (space_fn)(uintptr_t)f[3], f_verify = (verify_fn)(uintptr_t)f[4];
    f_rope = (rope_fn)(uintptr_t)f[5], f_paged = (paged_fn)(uintptr_t)f[6], f_paged_space = (paged_space_fn)(uintptr_t)f[7];
    f_prompt = (prompt_fn)(uintptr_t)f[8], f_prompt_space = (prompt_space_fn)(uintptr_t)f[9];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", py_setup, METH_VARARGS, NULL},
                                {"rows", (PyCFunction)(void (*)(void))py_rows, METH_FASTCALL, NULL},
                                {"keep", py_keep, METH_VARARGS, NULL},
                                {"release", py_release, METH_NOARGS, NULL},
                                {"attn", (PyCFunction)(void (*)(void))py_attn, METH_FASTCALL, NULL},
                                {"verify", (PyCFunction)(void (*)(void))py_verify, METH_FASTCALL, NULL},
                                {"paged", (PyCFunction)(void (*)(void))py_paged, METH_FASTCALL, NULL},
                                {"prompt", (PyCFunction)(void (*)(void))py_prompt, METH_FASTCALL, NULL},
                                {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qd_ops", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__qd_ops(void) {
    s_shape = PyUnicode_InternFromString("shape"), s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype"), s_ptr = PyUnicode_InternFromString("data_ptr");
    s_device = PyUnicode_InternFromString("get_device"), s_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_shape || !s_stride || !s_dtype || !s_ptr || !s_device || !s_stream) return NULL;
    return PyModule_Create(&module);
}
