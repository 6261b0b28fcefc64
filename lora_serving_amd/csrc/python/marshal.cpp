// Argument marshalling of the attention step's calls for the Python binding (mlora.py): torch tensors
// are checked and turned into device pointers through torch's tensor API, and the C entry point of the
// same name is called.  In Python the same checks cost 2 to 4 us a call, as much as a launch (cache_read
// 5.7 us a call against 3.7 here, qk_rope 8.0 against 3.8).  A call returns the entry point's status;
// tensors of another dtype, shape or device raise ValueError before it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mlora.h"

namespace {

using at::ScalarType;

[[noreturn]] void fail(const char *name, const std::string &what) { throw std::invalid_argument(std::string(name) + " " + what); }

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        fail(name, "must be a device tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda())
        fail(name, "must be a device tensor");
    return t;
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw std::runtime_error("");           // (the Python error stands)
    return v;
}

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw std::runtime_error("");
    return v;
}

int32_t int32(PyObject *o, const char *name)
{
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX)
        fail(name, "does not fit 32 bits");
    return (int32_t)v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw std::runtime_error("");
    return v != 0;
}

void *pointer(PyObject *o)
{
    void *p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred())
        throw std::runtime_error("");
    return p;
}

template <class T> const T *address(PyObject *o) { return o == Py_None ? nullptr : (const T *)pointer(o); }
hipStream_t stream(PyObject *o) { return (hipStream_t)pointer(o); }

void *dense(PyObject *o, const char *name, ScalarType type, const char *type_name)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type)
        fail(name, std::string("must have dtype ") + type_name);
    if (!t.is_contiguous())
        fail(name, "must be contiguous");
    return t.data_ptr();
}

// contiguous int32 of n values
const int32_t *ints(PyObject *o, const char *name, int64_t n)
{
    const int32_t *p = (const int32_t *)dense(o, name, ScalarType::Int, "int32");
    const int64_t has = THPVariable_Unpack(o).numel();
    if (has != n)
        fail(name, "has " + std::to_string(has) + " values, expected " + std::to_string(n));
    return p;
}

// bf16 [n][heads][head_dim] whose rows may lie apart
struct Rows {
    void *p;
    int64_t n, heads, d, stride;
};

Rows rows(PyObject *o, const char *name, const Rows *like = nullptr)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != ScalarType::BFloat16 || t.dim() != 3)
        fail(name, "must be bf16 [T][heads][head_dim]");
    Rows r{t.data_ptr(), t.size(0), t.size(1), t.size(2), 0};
    if (like && (r.n != like->n || r.heads != like->heads || r.d != like->d))
        fail(name, "has shape (" + std::to_string(r.n) + ", " + std::to_string(r.heads) + ", " + std::to_string(r.d) + "), expected (" +
                       std::to_string(like->n) + ", " + std::to_string(like->heads) + ", " + std::to_string(like->d) + ")");
    if (r.n > 0 && (t.stride(2) != 1 || (r.heads > 1 && t.stride(1) != r.d)))
        fail(name, "must hold contiguous heads in a row");
    r.stride = r.n > 1 ? t.stride(0) : r.heads * r.d;
    return r;
}

float *lse_of(PyObject *o, int64_t n, int64_t heads)
{
    if (o == Py_None)
        return nullptr;
    float *p = (float *)dense(o, "lse", ScalarType::Float, "float32");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != 2 || t.size(0) != n || t.size(1) != heads)
        fail("lse", "must have shape (" + std::to_string(n) + ", " + std::to_string(heads) + ")");
    return p;
}

const void *weight(PyObject *o, const char *name, int64_t d)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = tensor(o, name);
    const ScalarType s = t.scalar_type();
    if (s != ScalarType::BFloat16 && s != ScalarType::Short && s != ScalarType::UInt16)
        fail(name, "must be bf16");
    if (!t.is_contiguous())
        fail(name, "must be contiguous");
    if (t.numel() != d)
        fail(name, "must hold head_dim values");
    return t.data_ptr();
}

// The entry point itself runs without the interpreter's lock, as ctypes calls do: a launch waits where the queue is
// full.  Its arguments have been taken from their objects, which the caller holds.
template <class Call> mlora_status unlocked(Call call)
{
    struct Released {
        PyThreadState *state = PyEval_SaveThread();
        ~Released() { PyEval_RestoreThread(state); }
    } released;
    return call();
}

// (qkv, n_q_heads, n_kv_heads, head_dim, pos, rope, q_out, k_out, q_weight, k_weight, eps, cache, slot, stream)
mlora_status qk_rope(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "qkv");
    const int32_t hq = int32(a[1], "n_q_heads"), hkv = int32(a[2], "n_kv_heads"), d = int32(a[3], "head_dim");
    if (x.scalar_type() != ScalarType::BFloat16 || x.dim() != 2)
        fail("qkv", "must be a bf16 [T][width] device tensor");
    const int64_t T = x.size(0), width = ((int64_t)hq + 2 * (int64_t)hkv) * d;
    if (x.size(1) != width || (T > 0 && x.stride(1) != 1))
        fail("qkv", "must hold " + std::to_string(width) + " contiguous values in a row");
    const Rows want_q{nullptr, T, hq, d, 0}, want_k{nullptr, T, hkv, d, 0};
    const Rows q = rows(a[6], "q_out", &want_q);
    Rows k{};
    if (a[7] != Py_None)
        k = rows(a[7], "k_out", &want_k);
    const void *const px = x.data_ptr(), *const qw = weight(a[8], "q_weight", d), *const kw = weight(a[9], "k_weight", d);
    const int64_t x_stride = T > 1 ? x.stride(0) : width;
    const int32_t *const pos = ints(a[4], "pos", T), *const slot = a[12] == Py_None ? nullptr : ints(a[12], "slot", T);
    const mlora_rope *const rope = address<mlora_rope>(a[5]);
    const mlora_cache *const cache = address<mlora_cache>(a[11]);
    const float eps = (float)real(a[10]);
    const hipStream_t s = stream(a[13]);
    return unlocked([&] {
        return mlora_qk_rope(px, T, x_stride, hq, hkv, d, pos, rope, qw, kw, eps, q.p, q.stride, k.p, k.stride, cache, slot, s);
    });
}

// (cache, slot, k, v, stream)
mlora_status cache_read(PyObject *const *a)
{
    const mlora_cache *c = address<mlora_cache>(a[0]);
    const int64_t T = tensor(a[1], "slot").numel();
    void *out[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
        if (a[2 + i] == Py_None)
            continue;
        const char *name = i ? "v" : "k";
        out[i] = dense(a[2 + i], name, ScalarType::BFloat16, "bf16");
        const at::Tensor &t = THPVariable_Unpack(a[2 + i]);
        if (t.dim() != 3 || t.size(0) != T || t.size(1) != c->n_kv_heads || t.size(2) != c->head_dim)
            fail(name, "must have shape (" + std::to_string(T) + ", " + std::to_string(c->n_kv_heads) + ", " + std::to_string(c->head_dim) + ")");
    }
    const int32_t *const slot = ints(a[1], "slot", T);
    const hipStream_t s = stream(a[4]);
    return unlocked([&] { return mlora_cache_read(c, slot, T, out[0], out[1], s); });
}

// (q, k, v, cu_q, out, cu_k, max_q, causal, window, scale, lse, stream)
mlora_status attention(PyObject *const *a)
{
    const Rows q = rows(a[0], "q"), k = rows(a[1], "k"), v = rows(a[2], "v", &k), out = rows(a[4], "out", &q);
    if (k.d != q.d)
        fail("k", "must have the head_dim of q");
    const int64_t n = tensor(a[3], "cu_q").numel() - 1;
    const int32_t *const cu_q = ints(a[3], "cu_q", n + 1), *const cu_k = a[5] == Py_None ? nullptr : ints(a[5], "cu_k", n + 1);
    const int64_t max_q = a[6] == Py_None ? q.n : integer(a[6]);
    const int32_t causal = truth(a[7]), window = int32(a[8], "window");
    const float scale = (float)real(a[9]);
    float *const lse = lse_of(a[10], q.n, q.heads);
    const hipStream_t s = stream(a[11]);
    return unlocked([&] {
        return mlora_attention(q.p, q.stride, k.p, k.stride, v.p, v.stride, q.n, k.n, (int32_t)n, cu_q, cu_k, (int32_t)q.heads,
                               (int32_t)k.heads, (int32_t)q.d, max_q, causal, window, scale, out.p, out.stride, lse, s);
    });
}

// (q, cache, page_table, cu_q, kv_len, out, max_q, max_kv, causal, window, scale, lse, ws, stream)
mlora_status paged_attention(PyObject *const *a)
{
    const Rows q = rows(a[0], "q"), out = rows(a[5], "out", &q);
    const mlora_cache *c = address<mlora_cache>(a[1]);
    if (q.d != c->head_dim)
        fail("q", "must have the head_dim of the cache");
    const int64_t n = tensor(a[4], "kv_len").numel();
    const at::Tensor &table = tensor(a[2], "page_table");
    if (table.dim() != 2 || table.size(0) != n)
        fail("page_table", "must be [n_seqs][pages]");
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (a[12] != Py_None) {
        const at::Tensor &w = tensor(a[12], "ws");
        if (!w.is_contiguous())
            fail("ws", "must be contiguous");
        ws = w.data_ptr();
        ws_bytes = w.nbytes();
    }
    const int32_t *const pages = ints(a[2], "page_table", table.numel()), *const cu_q = ints(a[3], "cu_q", n + 1),
                  *const kv_len = ints(a[4], "kv_len", n);
    const int64_t width = table.size(1), max_q = integer(a[6]), max_kv = integer(a[7]);
    const int32_t causal = truth(a[8]), window = int32(a[9], "window");
    const float scale = (float)real(a[10]);
    float *const lse = lse_of(a[11], q.n, q.heads);
    const hipStream_t s = stream(a[13]);
    return unlocked([&] {
        return mlora_paged_attention(q.p, q.stride, q.n, (int32_t)q.heads, c, pages, width, (int32_t)n, cu_q, kv_len, max_q, max_kv,
                                     causal, window, scale, out.p, out.stride, lse, ws, ws_bytes, s);
    });
}

// no C++ exception leaves a call
template <mlora_status (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N)
        return PyErr_Format(PyExc_TypeError, "expected %d arguments", N);
    try {
        return PyLong_FromLong((long)F(args));
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define METHOD(name, f, n) {name, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("qk_rope", qk_rope, 14), METHOD("cache_read", cache_read, 5), METHOD("attention", attention, 12),
                         METHOD("paged_attention", paged_attention, 14), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
