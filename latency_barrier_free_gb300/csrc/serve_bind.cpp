// serve_bind.cpp -- the operators of rra_serve.h as a CPython module: takes
// torch tensors, checks them, fills in the argument structures and calls
// librra.so.  A call of these operators may run a microsecond on the GPU, so
// what the host does for it counts: head norms and rotation of 4 tokens took
// 8.9 us a call with the checks in Python, 5.7 with the tensors' attributes
// read through their Python objects, and 2.7 reading the tensors themselves.
// serve.py holds the public functions.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include "rra_serve.h"

namespace {

template <typename Args>
using Operator = rra_status_t (*)(const Args*, rra_stream_t);
Operator<rra_slot_map_args_t> fn_slot_map;
Operator<rra_qk_norm_rope_args_t> fn_rope;
Operator<rra_kv_tokens_args_t> fn_append, fn_read;
Operator<rra_kv_attention_args_t> fn_attention;
PyObject* s_cuda_stream;

struct Refused {};  // thrown with a Python exception set

[[noreturn]] void refuse(PyObject* type, const char* format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw Refused{};
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

// Refuses a GPU that is not the current one: a kernel would run on that one, with this one's addresses.
int on_current(int device) {
    const int now = (int)c10::cuda::current_device();
    if (device != now) refuse(PyExc_ValueError, "tensors on cuda:%d, but the current GPU is cuda:%d", device, now);
    return device;
}

// A tensor's GPU, the current one; refuses what is on none.
int device_of(const char* name, const at::Tensor& t) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return on_current((int)t.get_device());
}

void check(const char* name, const at::Tensor& t, at::ScalarType type, int device, bool fine, const char* what) {
    if (fine && t.scalar_type() == type && t.is_cuda() && t.get_device() == device) return;
    refuse(PyExc_ValueError, "%s must be a %s tensor, %s, on cuda:%d", name, c10::toString(type), what, device);
}

// Pointer of a contiguous tensor of at least n elements.
template <typename T>
T* flat(const char* name, const at::Tensor& t, at::ScalarType type, int64_t n, int device) {
    check(name, t, type, device, t.is_contiguous() && t.numel() >= n, "contiguous and large enough");
    return (T*)t.data_ptr();
}
template <typename T>
T* flat(const char* name, PyObject* o, at::ScalarType type, int64_t n, int device) {
    return flat<T>(name, tensor(name, o), type, n, device);
}

// Pointer and strides of a [tokens, heads, channels] tensor with adjacent channels.
void* rows(const char* name, const at::Tensor& t, at::ScalarType type, c10::IntArrayRef shape, int device, int64_t* token,
           int64_t* head) {
    check(name, t, type, device, t.dim() == 3 && t.sizes() == shape && (t.stride(2) == 1 || shape[2] <= 1),
          "[tokens, heads, channels] of the call's sizes with adjacent channels");
    // strides of a dimension of one element are never used
    *token = shape[0] > 1 ? t.stride(0) : shape[1] * shape[2] * 16;
    *head = shape[1] > 1 ? t.stride(1) : shape[2];
    return t.data_ptr();
}

int32_t* table_of(PyObject* o, int64_t requests, int device, int64_t* stride, int32_t* width) {
    const at::Tensor& t = tensor("block_table", o);
    check("block_table", t, at::kInt, device,
          t.dim() == 2 && t.size(0) == requests && t.size(1) <= INT32_MAX && (t.stride(1) == 1 || t.size(1) <= 1 || requests == 0),
          "[requests, pages] with adjacent pages");
    *stride = requests > 1 ? t.stride(0) : t.size(1);
    *width = (int32_t)t.size(1);
    return (int32_t*)t.data_ptr();
}

rra_stream_t stream_of(PyObject* o, int device) {
    if (o == Py_None) return (rra_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    PyObject* number = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttr(o, s_cuda_stream);
    if (number == nullptr) throw Refused{};
    void* s = PyLong_AsVoidPtr(number);
    Py_DECREF(number);
    if (s == nullptr && PyErr_Occurred()) throw Refused{};
    return (rra_stream_t)s;
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
int32_t integer32(PyObject* o) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_OverflowError, "argument does not fit 32 bits");
    return (int32_t)v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

void arguments(Py_ssize_t have, Py_ssize_t want) {
    if (have != want) refuse(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
}

int32_t value_dtype(at::ScalarType t) {
    if (t != at::kFloat && t != at::kBFloat16) refuse(PyExc_TypeError, "unsupported dtype (float32, bfloat16)");
    return t == at::kFloat ? RRA_FP32 : RRA_BF16;
}

// ------------------------------------------------------------- operators ----
long slot_map(PyObject* const* v, Py_ssize_t n) {
    arguments(n, 13);
    rra_slot_map_args_t a = {};
    const at::Tensor &seq = tensor("seq_len", v[0]), &free_pages = tensor("free_pages", v[3]), &slots = tensor("slots", v[8]);
    const int dev = device_of("seq_len", seq);
    const int64_t requests = seq.numel();
    a.seq_len = flat<int32_t>("seq_len", seq, at::kInt, 0, dev);
    a.new_len = flat<int32_t>("new_len", v[1], at::kInt, requests, dev);
    a.block_table = table_of(v[2], requests, dev, &a.table_stride, &a.table_pages);
    a.free_pages = flat<int32_t>("free_pages", free_pages, at::kInt, 0, dev);
    a.free_count = flat<int32_t>("free_count", v[4], at::kInt, 1, dev);
    a.page_tokens = integer32(v[5]);
    a.kv_len = flat<int32_t>("kv_len", v[6], at::kInt, requests, dev);
    a.cu_new = flat<int32_t>("cu_new", v[7], at::kInt, requests + 1, dev);
    a.slots = flat<int64_t>("slots", slots, at::kLong, 0, dev);
    a.tokens = slots.numel();
    a.positions = flat<int32_t>("positions", v[9], at::kInt, a.tokens, dev);
    a.free_left = flat<int32_t>("free_left", v[10], at::kInt, 1, dev);
    a.pages_short = flat<int32_t>("pages_short", v[11], at::kInt, 1, dev);
    if (requests > RRA_SERVE_MAX_REQUESTS || free_pages.numel() > INT32_MAX) return RRA_ERR_INVALID_ARG;
    a.requests = (int32_t)requests;
    a.num_pages = (int32_t)free_pages.numel();
    return fn_slot_map(&a, stream_of(v[12], dev));
}

long qk_norm_rope(PyObject* const* v, Py_ssize_t n) {
    arguments(n, 12);
    rra_qk_norm_rope_args_t a = {};
    const at::Tensor &q = tensor("q", v[0]), &k = tensor("k", v[1]);
    const int dev = device_of("q", q);
    const at::ScalarType type = q.scalar_type();
    a.dtype = value_dtype(type);
    if (q.dim() != 3 || k.dim() != 3 || q.size(0) != k.size(0) || q.size(2) != k.size(2) || q.size(1) > INT32_MAX ||
        k.size(1) > INT32_MAX || q.size(2) > INT32_MAX)
        refuse(PyExc_ValueError, "q and k must be [tokens, heads, channels] with the same tokens and channels");
    a.tokens = q.size(0);
    a.q_heads = (int32_t)q.size(1);
    a.k_heads = (int32_t)k.size(1);
    a.head_dim = (int32_t)q.size(2);
    a.q = rows("q", q, type, q.sizes(), dev, &a.q_token_stride, &a.q_head_stride);
    a.k = rows("k", k, type, k.sizes(), dev, &a.k_token_stride, &a.k_head_stride);
    a.q_out = rows("q_out", tensor("q_out", v[7]), type, q.sizes(), dev, &a.q_out_token_stride, &a.q_out_head_stride);
    a.k_out = rows("k_out", tensor("k_out", v[8]), type, k.sizes(), dev, &a.k_out_token_stride, &a.k_out_head_stride);
    if (v[2] != Py_None) a.q_weight = flat<void>("q_weight", v[2], type, a.head_dim, dev);
    if (v[3] != Py_None) a.k_weight = flat<void>("k_weight", v[3], type, a.head_dim, dev);
    if (v[4] != Py_None) {
        const at::Tensor &cos = tensor("cos", v[4]), &sin = tensor("sin", v[5]);
        if (cos.dim() != 2 || cos.sizes() != sin.sizes() || cos.size(1) > a.head_dim)
            refuse(PyExc_ValueError, "cos and sin must be [max_position, rot/2]");
        a.cos = flat<float>("cos", cos, at::kFloat, 0, dev);
        a.sin = flat<float>("sin", sin, at::kFloat, 0, dev);
        a.positions = flat<int32_t>("positions", v[6], at::kInt, a.tokens, dev);
        a.max_position = cos.size(0);
        a.rot = (int32_t)(2 * cos.size(1));
    }
    a.eps = real(v[9]);
    a.interleaved = truth(v[10]);
    return fn_rope(&a, stream_of(v[11], dev));
}

// The first argument of a cache's calls: its structure, as bytes.
rra_kv_cache_t cache_of(PyObject* bytes) {
    rra_kv_cache_t c;
    if (!PyBytes_Check(bytes) || PyBytes_GET_SIZE(bytes) != (Py_ssize_t)sizeof c) refuse(PyExc_TypeError, "expected a cache");
    memcpy(&c, PyBytes_AS_STRING(bytes), sizeof c);
    return c;
}

// (cache, device, k, v, slots, stream)
long kv_tokens(PyObject* const* v, Py_ssize_t n, Operator<rra_kv_tokens_args_t> fn) {
    arguments(n, 6);
    rra_kv_tokens_args_t a = {};
    a.cache = cache_of(v[0]);
    const int dev = on_current(integer32(v[1]));
    const at::Tensor &k = tensor("k", v[2]), &slots = tensor("slots", v[4]);
    const at::ScalarType type = k.scalar_type();
    a.dtype = value_dtype(type);
    a.slots = flat<int64_t>("slots", slots, at::kLong, 0, dev);
    a.tokens = slots.numel();
    const int64_t shape[3] = {a.tokens, a.cache.kv_heads, a.cache.head_dim};
    a.k = rows("k", k, type, shape, dev, &a.k_token_stride, &a.k_head_stride);
    a.v = rows("v", tensor("v", v[3]), type, shape, dev, &a.v_token_stride, &a.v_head_stride);
    return fn(&a, stream_of(v[5], dev));
}
long kv_append(PyObject* const* v, Py_ssize_t n) { return kv_tokens(v, n, fn_append); }
long kv_read(PyObject* const* v, Py_ssize_t n) { return kv_tokens(v, n, fn_read); }

// (cache, device, workspace, q, out, cu_q, kv_len, block_table, max_q, max_kv, scale, causal, window, lse, stream, the
// workspace's own stream)
long kv_attention(PyObject* const* v, Py_ssize_t n) {
    arguments(n, 16);
    rra_kv_attention_args_t a = {};
    a.cache = cache_of(v[0]);
    const int dev = on_current(integer32(v[1]));
    const at::Tensor &q = tensor("q", v[3]), &kv = tensor("kv_len", v[6]);
    if (q.dim() != 3 || q.size(2) != a.cache.head_dim || q.size(1) < 1 || q.size(1) % a.cache.kv_heads != 0 || q.size(1) > INT32_MAX)
        refuse(PyExc_ValueError, "q must be [tokens, heads, %d], heads a multiple of %d", a.cache.head_dim, a.cache.kv_heads);
    const at::Tensor& workspace = tensor("workspace", v[2]);
    a.workspace = workspace.data_ptr();
    a.tokens = q.size(0);
    a.q_heads = (int32_t)q.size(1);
    a.q = rows("q", q, at::kBFloat16, q.sizes(), dev, &a.q_token_stride, &a.q_head_stride);
    a.out = rows("out", tensor("out", v[4]), at::kBFloat16, q.sizes(), dev, &a.out_token_stride, &a.out_head_stride);
    const int64_t requests = kv.numel();
    a.kv_len = flat<int32_t>("kv_len", kv, at::kInt, 0, dev);
    a.cu_q = flat<int32_t>("cu_q", v[5], at::kInt, requests + 1, dev);
    a.block_table = table_of(v[7], requests, dev, &a.table_stride, &a.table_pages);
    a.max_q = integer32(v[8]);
    a.max_kv = integer32(v[9]);
    a.scale = real(v[10]);
    a.causal = truth(v[11]);
    a.window = integer32(v[12]);
    if (v[13] != Py_None) a.lse = flat<float>("lse", v[13], at::kFloat, a.tokens * a.q_heads, dev);
    if (requests > RRA_SERVE_MAX_REQUESTS) return RRA_ERR_INVALID_ARG;
    a.requests = (int32_t)requests;
    const rra_stream_t stream = stream_of(v[14], dev);
    // The caller does not know the workspace: its memory must not go to another tensor before this call's work is done.  (Of a
    // stream given by its number nothing is known, not even whether it still exists then: there the caller keeps the cache.)
    if (stream != (rra_stream_t)PyLong_AsVoidPtr(v[15]) && !PyLong_Check(v[14]))
        c10::cuda::CUDACachingAllocator::recordStream(workspace.storage().data_ptr(),
                                                      c10::cuda::getStreamFromExternal((cudaStream_t)stream, (c10::DeviceIndex)dev));
    return fn_attention(&a, stream);
}

// ---------------------------------------------------------------- module ----
// init(path of librra.so)
long init(PyObject* const* v, Py_ssize_t n) {
    arguments(n, 1);
    const char* path = PyUnicode_AsUTF8(v[0]);
    if (path == nullptr) throw Refused{};
    void* lib = dlopen(path, RTLD_NOW);
    if (lib == nullptr) refuse(PyExc_RuntimeError, "%s", dlerror());
    auto find = [&](auto& fn, const char* name) {
        fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(dlsym(lib, name));
        if (fn == nullptr) refuse(PyExc_RuntimeError, "librra.so lacks %s: build it again", name);
    };
    find(fn_slot_map, "rra_slot_map");
    find(fn_rope, "rra_qk_norm_rope");
    find(fn_append, "rra_kv_append");
    find(fn_read, "rra_kv_read");
    find(fn_attention, "rra_kv_attention");
    return 0;
}

// A function of this module: its status as a number.  No C++ exception leaves it.
template <long (*F)(PyObject* const*, Py_ssize_t)>
PyObject* call(PyObject*, PyObject* const* v, Py_ssize_t n) {
    try {
        return PyLong_FromLong(F(v, n));
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <long (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)())call<F>, METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<init>("init"),           method<slot_map>("slot_map"),  method<qk_norm_rope>("qk_norm_rope"),
                         method<kv_append>("kv_append"), method<kv_read>("kv_read"),    method<kv_attention>("kv_attention"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) {
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    return s_cuda_stream == nullptr ? nullptr : PyModule_Create(&module);
}
