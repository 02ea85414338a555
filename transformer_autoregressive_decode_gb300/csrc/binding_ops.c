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

static rows_fn f_append, f_read;
static attn_fn f_attn;
static space_fn f_space;
static verify_fn f_verify;
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

/* n contiguous int32 values, or None */
static int read_ints(PyObject *t, int64_t n, const int32_t **to, const char *what) {
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
    if (!ok || count != n) {
        PyErr_Format(PyExc_ValueError, "%s must be %lld contiguous int32 values", what, (long long)n);
        return 0;
    }
    *to = (const int32_t *)x.ptr;
    return 1;
}

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
    if (PyErr_Occurred() || !read_tensor(a[0], &q) || !read_tensor(a[3], &o)) return NULL;
    const int64_t D = c->head_dim, B = c->n_streams;
    if (q.nd != 4 || o.nd != 4 || q.type != o.type || q.shape[0] != B || q.shape[3] != D || o.shape[0] != B ||
        o.shape[1] != q.shape[1] || o.shape[2] != q.shape[2] || o.shape[3] != D) {
        PyErr_Format(PyExc_ValueError, "q and out must be [%d, tokens, q_heads, %d] of one type", c->n_streams, c->head_dim);
        return NULL;
    }
    if (q.stride[3] != 1 || o.stride[3] != 1 || (q.shape[2] > 1 && (q.stride[2] != D || o.stride[2] != D))) {
        bad("the heads of q and out must be contiguous");
        return NULL;
    }
    if (!fits(&q) || !type_of(&q, &dtype) || !opt_int(a[5], c->smax, &most) || !opt_int(a[8], p ? p->smax : 0, &plen))
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
    double scale = 1.0 / (D == 64 ? 8.0 : 11.313708498984761);   /* head_dim ** -0.5 */
    if (a[6] != Py_None) {
        scale = PyFloat_AsDouble(a[6]);
        if (scale == -1.0 && PyErr_Occurred()) return NULL;
    }
    if (!read_ints(a[2], B, &lengths, "lengths") || !read_ints(a[4], B, &n_new, "n_new") || !stream_of(a[11], a[0], &s, &dev))
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
            int i = n_scratch;
            if (dev >= 0) {
                PyObject *cap = PyObject_CallNoArgs(capturing);
                if (!cap) return NULL;
                const int is = PyObject_IsTrue(cap);
                Py_DECREF(cap);
                for (i = 0; !is && i < n_scratch; ++i)
                    if (scratch[i].dev == dev && scratch[i].stream == s && scratch[i].size >= need) break;
                if (is) i = n_scratch;
            }
            if (i == n_scratch) return PyLong_FromSize_t(need);
            ws = scratch[i].ptr, have = scratch[i].size;
        }
    }
    return PyLong_FromLong(f_attn(c, p, plen, q.ptr, B > 1 ? q.stride[0] : 0, T > 1 ? q.stride[1] : 0, o.ptr,
                                  B > 1 ? o.stride[0] : 0, T > 1 ? o.stride[1] : 0, dtype, T, QH, (float)scale, lengths,
                                  n_new, most, ws, have, s));
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

/* setup(append, read, attn, workspace, verify: addresses; float32, bfloat16, int32, current raw stream, whether it is being
 * captured: torch's) */
static PyObject *py_setup(PyObject *self, PyObject *args) {
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "KKKKKOOOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &t_f32, &t_bf16, &t_i32, &raw_stream,
                          &capturing))
        return NULL;
    Py_INCREF(t_f32), Py_INCREF(t_bf16), Py_INCREF(t_i32), Py_INCREF(raw_stream), Py_INCREF(capturing);
    f_append = (rows_fn)(uintptr_t)f[0], f_read = (rows_fn)(uintptr_t)f[1], f_attn = (attn_fn)(uintptr_t)f[2];
    f_space = (space_fn)(uintptr_t)f[3], f_verify = (verify_fn)(uintptr_t)f[4];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", py_setup, METH_VARARGS, NULL},
                                {"rows", (PyCFunction)(void (*)(void))py_rows, METH_FASTCALL, NULL},
                                {"keep", py_keep, METH_VARARGS, NULL},
                                {"release", py_release, METH_NOARGS, NULL},
                                {"attn", (PyCFunction)(void (*)(void))py_attn, METH_FASTCALL, NULL},
                                {"verify", (PyCFunction)(void (*)(void))py_verify, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qd_ops", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__qd_ops(void) {
    s_shape = PyUnicode_InternFromString("shape"), s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype"), s_ptr = PyUnicode_InternFromString("data_ptr");
    s_device = PyUnicode_InternFromString("get_device"), s_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_shape || !s_stride || !s_dtype || !s_ptr || !s_device || !s_stream) return NULL;
    return PyModule_Create(&module);
}
