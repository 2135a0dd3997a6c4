/* serve_bind.c -- the operators of rra_serve.h as a CPython module: takes
 * torch tensors, checks them, fills in the argument structures and calls
 * librra.so.  A call of these operators may run a microsecond on the GPU, and
 * the checks written in Python took five (head norms and rotation of 4 tokens:
 * 8.9 us a call); they are the same here.
 *
 * Only attributes that every tensor has are used (dtype, shape, stride(),
 * data_ptr(), get_device(), ...), through the Python objects, so nothing here
 * depends on torch's own headers.  serve.py holds the public functions. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include "rra_serve.h"

static rra_status_t (*fn_slot_map)(const rra_slot_map_args_t*, rra_stream_t);
static rra_status_t (*fn_rope)(const rra_qk_norm_rope_args_t*, rra_stream_t);
static rra_status_t (*fn_append)(const rra_kv_tokens_args_t*, rra_stream_t);
static rra_status_t (*fn_read)(const rra_kv_tokens_args_t*, rra_stream_t);
static rra_status_t (*fn_attention)(const rra_kv_attention_args_t*, rra_stream_t);

static PyObject *s_data_ptr, *s_get_device, *s_dtype, *s_shape, *s_stride, *s_is_contiguous, *s_numel, *s_cuda_stream;
static PyObject *t_float32, *t_bfloat16, *t_int32, *t_int64, *current_stream;

/* ------------------------------------------------------------- tensors ---- */
static int as_int64(PyObject* o, int64_t* v) { /* takes the reference */
    if (o == NULL) return -1;
    *v = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

static int call_int(PyObject* t, PyObject* method, int64_t* v) { return as_int64(PyObject_CallMethodNoArgs(t, method), v); }

static int pointer(PyObject* t, void** p) {
    PyObject* o = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (o == NULL) return -1;
    *p = (void*)PyLong_AsUnsignedLongLong(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

/* Whether t's dtype is `dtype`: 1, 0, or -1 with an exception. */
static int has_dtype(PyObject* t, PyObject* dtype) {
    PyObject* o = PyObject_GetAttr(t, s_dtype);
    if (o == NULL) return -1;
    Py_DECREF(o);
    return o == dtype;
}

static int refuse(const char* name, PyObject* dtype, const char* what, int64_t device) {
    PyErr_Format(PyExc_ValueError, "%s must be a %S tensor, %s, on cuda:%lld", name, dtype, what, (long long)device);
    return -1;
}

/* Sizes of a tuple (a shape, or strides) of n entries. */
static int sizes(PyObject* tuple, int n, int64_t* v) { /* takes the reference */
    if (tuple == NULL) return -1;
    if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != n) {
        Py_DECREF(tuple);
        PyErr_Format(PyExc_ValueError, "expected a tensor of %d dimensions", n);
        return -1;
    }
    for (int i = 0; i < n; ++i) v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    Py_DECREF(tuple);
    return PyErr_Occurred() ? -1 : 0;
}
static int shape_of(PyObject* t, int n, int64_t* v) { return sizes(PyObject_GetAttr(t, s_shape), n, v); }
static int stride_of(PyObject* t, int n, int64_t* v) { return sizes(PyObject_CallMethodNoArgs(t, s_stride), n, v); }

/* A tensor's GPU; refuses what is on none. */
static int device_of(PyObject* t, int64_t* device) {
    if (call_int(t, s_get_device, device) < 0) return -1;
    if (*device < 0) {
        PyErr_SetString(PyExc_ValueError, "expected CUDA tensors");
        return -1;
    }
    return 0;
}
static int on(PyObject* t, PyObject* dtype, int64_t device) { /* 1, 0, or -1 */
    const int same = has_dtype(t, dtype);
    if (same <= 0) return same;
    int64_t d;
    if (call_int(t, s_get_device, &d) < 0) return -1;
    return d == device;
}

/* Pointer of a contiguous tensor of at least n elements; their number, if asked. */
static int flat(const char* name, PyObject* t, PyObject* dtype, int64_t n, int64_t device, void** p, int64_t* count) {
    const int fine = on(t, dtype, device);
    if (fine < 0) return -1;
    int64_t have;
    if (call_int(t, s_numel, &have) < 0) return -1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (c == NULL) return -1;
    Py_DECREF(c);
    if (!fine || c != Py_True || have < n) {
        char what[64];
        snprintf(what, sizeof what, "contiguous, of at least %lld elements", (long long)n);
        return refuse(name, dtype, what, device);
    }
    if (count != NULL) *count = have;
    return pointer(t, p);
}

/* Pointer and strides of a [tokens, heads, channels] tensor with adjacent channels. */
static int rows(const char* name, PyObject* t, PyObject* dtype, const int64_t* shape, int64_t device, void** p,
                int64_t* token, int64_t* head) {
    const int fine = on(t, dtype, device);
    if (fine < 0) return -1;
    int64_t have[3], stride[3];
    if (shape_of(t, 3, have) < 0 || stride_of(t, 3, stride) < 0) return -1;
    if (!fine || have[0] != shape[0] || have[1] != shape[1] || have[2] != shape[2] || (stride[2] != 1 && shape[2] > 1)) {
        char what[128];
        snprintf(what, sizeof what, "of shape (%lld, %lld, %lld) with adjacent channels", (long long)shape[0],
                 (long long)shape[1], (long long)shape[2]);
        return refuse(name, dtype, what, device);
    }
    /* strides of a dimension of one element are never used */
    *token = shape[0] > 1 ? stride[0] : shape[1] * shape[2] * 16;
    *head = shape[1] > 1 ? stride[1] : shape[2];
    return pointer(t, p);
}

static int table_of(PyObject* t, int64_t requests, int64_t device, int32_t** p, int64_t* stride, int32_t* width) {
    const int fine = on(t, t_int32, device);
    if (fine < 0) return -1;
    int64_t have[2], step[2];
    if (shape_of(t, 2, have) < 0 || stride_of(t, 2, step) < 0) return -1;
    if (!fine || have[0] != requests || have[1] > INT32_MAX || (step[1] != 1 && have[1] > 1 && have[0] > 0))
        return refuse("block_table", t_int32, "[requests, pages] with adjacent pages", device);
    *stride = have[0] > 1 ? step[0] : have[1];
    *width = (int32_t)have[1];
    return pointer(t, (void**)p);
}

static int stream_of(PyObject* stream, int64_t device, rra_stream_t* s) {
    PyObject* o;
    if (stream == Py_None) {
        PyObject* d = PyLong_FromLongLong(device);
        if (d == NULL) return -1;
        o = PyObject_CallOneArg(current_stream, d);
        Py_DECREF(d);
    } else if (PyLong_Check(stream)) {
        o = Py_NewRef(stream);
    } else {
        o = PyObject_GetAttr(stream, s_cuda_stream);
    }
    if (o == NULL) return -1;
    *s = (rra_stream_t)PyLong_AsUnsignedLongLong(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

static int arg_int32(PyObject* o, int32_t* v) {
    int64_t x;
    Py_INCREF(o);
    if (as_int64(o, &x) < 0) return -1;
    if (x < INT32_MIN || x > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
        return -1;
    }
    *v = (int32_t)x;
    return 0;
}

static int arg_count(Py_ssize_t have, Py_ssize_t want) {
    if (have == want) return 0;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
    return -1;
}

static int value_dtype(PyObject* t, PyObject** dtype, int32_t* code) {
    const int f = has_dtype(t, t_float32), b = f == 0 ? has_dtype(t, t_bfloat16) : 0;
    if (f < 0 || b < 0) return -1;
    if (!f && !b) {
        PyErr_SetString(PyExc_TypeError, "unsupported dtype (float32, bfloat16)");
        return -1;
    }
    *dtype = f ? t_float32 : t_bfloat16;
    *code = f ? RRA_FP32 : RRA_BF16;
    return 0;
}

/* ------------------------------------------------------------ operators ---- */
static PyObject* slot_map(PyObject* self, PyObject* const* v, Py_ssize_t n) {
    (void)self;
    rra_slot_map_args_t a = {0};
    int64_t dev, requests, pages;
    rra_stream_t stream;
    if (arg_count(n, 13) < 0 || device_of(v[0], &dev) < 0 || call_int(v[0], s_numel, &requests) < 0 ||
        flat("seq_len", v[0], t_int32, 0, dev, (void**)&a.seq_len, NULL) < 0 ||
        flat("new_len", v[1], t_int32, requests, dev, (void**)&a.new_len, NULL) < 0 ||
        table_of(v[2], requests, dev, &a.block_table, &a.table_stride, &a.table_pages) < 0 ||
        flat("free_pages", v[3], t_int32, 0, dev, (void**)&a.free_pages, &pages) < 0 ||
        flat("free_count", v[4], t_int32, 1, dev, (void**)&a.free_count, NULL) < 0 || arg_int32(v[5], &a.page_tokens) < 0 ||
        flat("kv_len", v[6], t_int32, requests, dev, (void**)&a.kv_len, NULL) < 0 ||
        flat("cu_new", v[7], t_int32, requests + 1, dev, (void**)&a.cu_new, NULL) < 0 ||
        flat("slots", v[8], t_int64, 0, dev, (void**)&a.slots, &a.tokens) < 0 ||
        flat("positions", v[9], t_int32, a.tokens, dev, (void**)&a.positions, NULL) < 0 ||
        flat("free_left", v[10], t_int32, 1, dev, (void**)&a.free_left, NULL) < 0 ||
        flat("pages_short", v[11], t_int32, 1, dev, (void**)&a.pages_short, NULL) < 0 || stream_of(v[12], dev, &stream) < 0)
        return NULL;
    if (requests > RRA_SERVE_MAX_REQUESTS || pages > INT32_MAX) return PyLong_FromLong(RRA_ERR_INVALID_ARG);
    a.requests = (int32_t)requests;
    a.num_pages = (int32_t)pages;
    return PyLong_FromLong(fn_slot_map(&a, stream));
}

static PyObject* qk_norm_rope(PyObject* self, PyObject* const* v, Py_ssize_t n) {
    (void)self;
    rra_qk_norm_rope_args_t a = {0};
    int64_t dev, q[3], k[3], cs[2], sn[2];
    PyObject* dt;
    rra_stream_t stream;
    if (arg_count(n, 12) < 0 || device_of(v[0], &dev) < 0 || value_dtype(v[0], &dt, &a.dtype) < 0 || shape_of(v[0], 3, q) < 0 ||
        shape_of(v[1], 3, k) < 0)
        return NULL;
    if (q[0] != k[0] || q[2] != k[2] || q[1] > INT32_MAX || k[1] > INT32_MAX || q[2] > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "q and k must be [tokens, heads, channels] with the same tokens and channels");
        return NULL;
    }
    if (rows("q", v[0], dt, q, dev, (void**)&a.q, &a.q_token_stride, &a.q_head_stride) < 0 ||
        rows("k", v[1], dt, k, dev, (void**)&a.k, &a.k_token_stride, &a.k_head_stride) < 0 ||
        rows("q_out", v[7], dt, q, dev, &a.q_out, &a.q_out_token_stride, &a.q_out_head_stride) < 0 ||
        rows("k_out", v[8], dt, k, dev, &a.k_out, &a.k_out_token_stride, &a.k_out_head_stride) < 0)
        return NULL;
    if (v[2] != Py_None && flat("q_weight", v[2], dt, q[2], dev, (void**)&a.q_weight, NULL) < 0) return NULL;
    if (v[3] != Py_None && flat("k_weight", v[3], dt, q[2], dev, (void**)&a.k_weight, NULL) < 0) return NULL;
    if (v[4] != Py_None) {
        if (shape_of(v[4], 2, cs) < 0 || shape_of(v[5], 2, sn) < 0) return NULL;
        if (cs[0] != sn[0] || cs[1] != sn[1] || cs[1] > q[2]) {
            PyErr_SetString(PyExc_ValueError, "cos and sin must be [max_position, rot/2]");
            return NULL;
        }
        if (flat("cos", v[4], t_float32, 0, dev, (void**)&a.cos, NULL) < 0 ||
            flat("sin", v[5], t_float32, 0, dev, (void**)&a.sin, NULL) < 0 ||
            flat("positions", v[6], t_int32, q[0], dev, (void**)&a.positions, NULL) < 0)
            return NULL;
        a.max_position = cs[0];
        a.rot = (int32_t)(2 * cs[1]);
    }
    a.eps = PyFloat_AsDouble(v[9]);
    a.interleaved = PyObject_IsTrue(v[10]);
    if (PyErr_Occurred() || stream_of(v[11], dev, &stream) < 0) return NULL;
    a.tokens = q[0];
    a.q_heads = (int32_t)q[1];
    a.k_heads = (int32_t)k[1];
    a.head_dim = (int32_t)q[2];
    return PyLong_FromLong(fn_rope(&a, stream));
}

/* The first arguments of a cache's calls: its structure, as bytes, and its GPU. */
static int cache_of(PyObject* bytes, PyObject* device, rra_kv_cache_t* c, int64_t* dev) {
    if (!PyBytes_Check(bytes) || PyBytes_GET_SIZE(bytes) != (Py_ssize_t)sizeof *c) {
        PyErr_SetString(PyExc_TypeError, "expected a cache");
        return -1;
    }
    memcpy(c, PyBytes_AS_STRING(bytes), sizeof *c);
    Py_INCREF(device);
    return as_int64(device, dev);
}

static PyObject* kv_tokens(PyObject* const* v, Py_ssize_t n, rra_status_t (*fn)(const rra_kv_tokens_args_t*, rra_stream_t)) {
    rra_kv_tokens_args_t a = {0};
    int64_t dev, shape[3];
    PyObject* dt;
    rra_stream_t stream;
    if (arg_count(n, 6) < 0 || cache_of(v[0], v[1], &a.cache, &dev) < 0 || value_dtype(v[2], &dt, &a.dtype) < 0 ||
        flat("slots", v[4], t_int64, 0, dev, (void**)&a.slots, &a.tokens) < 0)
        return NULL;
    shape[0] = a.tokens;
    shape[1] = a.cache.kv_heads;
    shape[2] = a.cache.head_dim;
    if (rows("k", v[2], dt, shape, dev, &a.k, &a.k_token_stride, &a.k_head_stride) < 0 ||
        rows("v", v[3], dt, shape, dev, &a.v, &a.v_token_stride, &a.v_head_stride) < 0 || stream_of(v[5], dev, &stream) < 0)
        return NULL;
    return PyLong_FromLong(fn(&a, stream));
}
static PyObject* kv_append(PyObject* self, PyObject* const* v, Py_ssize_t n) {
    (void)self;
    return kv_tokens(v, n, fn_append);
}
static PyObject* kv_read(PyObject* self, PyObject* const* v, Py_ssize_t n) {
    (void)self;
    return kv_tokens(v, n, fn_read);
}

/* (cache, device, workspace's address, q, out, cu_q, kv_len, block_table, max_q, max_kv, scale, causal, window, lse, stream) */
static PyObject* kv_attention(PyObject* self, PyObject* const* v, Py_ssize_t n) {
    (void)self;
    rra_kv_attention_args_t a = {0};
    int64_t dev, q[3], requests, workspace;
    rra_stream_t stream;
    if (arg_count(n, 15) < 0 || cache_of(v[0], v[1], &a.cache, &dev) < 0 || shape_of(v[3], 3, q) < 0) return NULL;
    if (q[2] != a.cache.head_dim || q[1] < 1 || q[1] % a.cache.kv_heads != 0 || q[1] > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "q must be [tokens, heads, %d], heads a multiple of %d", a.cache.head_dim, a.cache.kv_heads);
        return NULL;
    }
    Py_INCREF(v[2]);
    if (as_int64(v[2], &workspace) < 0 ||
        rows("q", v[3], t_bfloat16, q, dev, (void**)&a.q, &a.q_token_stride, &a.q_head_stride) < 0 ||
        rows("out", v[4], t_bfloat16, q, dev, &a.out, &a.out_token_stride, &a.out_head_stride) < 0 ||
        flat("kv_len", v[6], t_int32, 0, dev, (void**)&a.kv_len, &requests) < 0 ||
        flat("cu_q", v[5], t_int32, requests + 1, dev, (void**)&a.cu_q, NULL) < 0 ||
        table_of(v[7], requests, dev, (int32_t**)&a.block_table, &a.table_stride, &a.table_pages) < 0 ||
        arg_int32(v[8], &a.max_q) < 0 || arg_int32(v[9], &a.max_kv) < 0 || arg_int32(v[12], &a.window) < 0)
        return NULL;
    if (v[13] != Py_None && flat("lse", v[13], t_float32, q[0] * q[1], dev, (void**)&a.lse, NULL) < 0) return NULL;
    a.workspace = (void*)(uintptr_t)workspace;
    a.scale = PyFloat_AsDouble(v[10]);
    a.causal = PyObject_IsTrue(v[11]);
    if (PyErr_Occurred() || stream_of(v[14], dev, &stream) < 0) return NULL;
    if (requests > RRA_SERVE_MAX_REQUESTS) return PyLong_FromLong(RRA_ERR_INVALID_ARG);
    a.requests = (int32_t)requests;
    a.tokens = q[0];
    a.q_heads = (int32_t)q[1];
    return PyLong_FromLong(fn_attention(&a, stream));
}

/* ---------------------------------------------------------------- module ---- */
/* init(path of librra.so, float32, bfloat16, int32, int64, current-stream function) */
static PyObject* init(PyObject* self, PyObject* const* v, Py_ssize_t n) {
    (void)self;
    if (arg_count(n, 6) < 0) return NULL;
    const char* path = PyUnicode_AsUTF8(v[0]);
    if (path == NULL) return NULL;
    void* lib = dlopen(path, RTLD_NOW);
    if (lib == NULL) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return NULL;
    }
    *(void**)&fn_slot_map = dlsym(lib, "rra_slot_map");
    *(void**)&fn_rope = dlsym(lib, "rra_qk_norm_rope");
    *(void**)&fn_append = dlsym(lib, "rra_kv_append");
    *(void**)&fn_read = dlsym(lib, "rra_kv_read");
    *(void**)&fn_attention = dlsym(lib, "rra_kv_attention");
    if (!fn_slot_map || !fn_rope || !fn_append || !fn_read || !fn_attention) {
        PyErr_SetString(PyExc_RuntimeError, "librra.so lacks an operator: build it again");
        return NULL;
    }
    t_float32 = Py_NewRef(v[1]);
    t_bfloat16 = Py_NewRef(v[2]);
    t_int32 = Py_NewRef(v[3]);
    t_int64 = Py_NewRef(v[4]);
    current_stream = Py_NewRef(v[5]);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, NULL},
    {"slot_map", (PyCFunction)(void (*)(void))slot_map, METH_FASTCALL, NULL},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, NULL},
    {"kv_read", (PyCFunction)(void (*)(void))kv_read, METH_FASTCALL, NULL},
    {"kv_attention", (PyCFunction)(void (*)(void))kv_attention, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__serve(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_numel = PyUnicode_InternFromString("numel");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    return PyErr_Occurred() ? NULL : PyModule_Create(&module);
}
