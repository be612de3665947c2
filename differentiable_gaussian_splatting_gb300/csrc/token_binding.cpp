// token_binding.cpp -- the Python binding of the token operators: checks torch tensors and
// passes plain pointers to the calls of include/gs.h.  What the package's Python code does
// for the other calls through ctypes is done here in C++, because these are called many
// times a training step on few tokens: on the GB300's Grace a call's host time is 3 to 4 us
// (6 for attention's gradient with its two launches) instead of 6 to 23.  Errors are those of
// the Python code: TypeError and ValueError for tensors; the status of the call is returned.
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <exception>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/gs.h"

namespace {

using at::Tensor;
using c10::ScalarType;

struct TypeError : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct ValueError : std::runtime_error {
    using std::runtime_error::runtime_error;
};

template <typename... A>
std::string text(const A&... a) {
    std::ostringstream s;
    (s << ... << a);
    return s.str();
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeError(text(name, ": expected a torch tensor"));
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) throw ValueError(text(name, ": must be a CUDA tensor"));
    return t;
}

void* address(const Tensor& t) { return t.numel() > 0 ? t.data_ptr() : nullptr; }

void want_type(const Tensor& t, const char* name, ScalarType type) {
    if (t.scalar_type() != type)
        throw ValueError(text(name, ": expected ", type, ", got ", t.scalar_type()));
}

// [tokens][heads][head_dim], contiguous in its last dimension; with `like`, of its shape
gs_heads heads(PyObject* o, const char* name, ScalarType type, const Tensor* like = nullptr) {
    const Tensor& t = tensor(o, name);
    if (t.dim() != 3)
        throw ValueError(text(name, ": expected [tokens, heads, head_dim], got ", t.sizes()));
    if (like && t.sizes() != like->sizes())
        throw ValueError(text(name, ": expected shape ", like->sizes(), ", got ", t.sizes()));
    want_type(t, name, type);
    if (t.stride(2) != 1 && t.size(2) > 1 && t.numel() > 0)
        throw ValueError(text(name, ": the last dimension must be contiguous"));
    return {address(t), t.stride(0), t.stride(1)};
}

// a contiguous tensor of at least n elements, or null where it may be None
void* flat(PyObject* o, const char* name, ScalarType type, int64_t n, bool optional = false) {
    if (o == Py_None) {
        if (optional) return nullptr;
        throw ValueError(text(name, " is required"));
    }
    const Tensor& t = tensor(o, name);
    want_type(t, name, type);
    if (!t.is_contiguous()) throw ValueError(text(name, ": must be contiguous"));
    if (t.numel() < n)
        throw ValueError(text(name, ": needs at least ", n, " elements, has ", t.numel()));
    return address(t);
}

// a contiguous tensor of exactly the shape of `like`, or null where it may be None
void* alike(PyObject* o, const char* name, const Tensor& like, bool optional = false) {
    void* p = flat(o, name, like.scalar_type(), 0, optional);
    if (o != Py_None && THPVariable_Unpack(o).sizes() != like.sizes())
        throw ValueError(text(name, ": expected shape ", like.sizes(), ", got ",
                              THPVariable_Unpack(o).sizes()));
    return p;
}

// head_dim values of fp32 (weights, which all heads share, or their gradient), or null for None
float* weights(PyObject* o, const char* name, int64_t dim) {
    void* p = flat(o, name, ScalarType::Float, dim, true);
    if (o != Py_None && THPVariable_Unpack(o).numel() != dim)
        throw ValueError(text(name, ": expected ", dim, " values, got ",
                              THPVariable_Unpack(o).sizes()));
    return static_cast<float*>(p);
}

struct Bytes {
    void* p;
    size_t n;
};
Bytes workspace(PyObject* o) {
    void* p = flat(o, "workspace", ScalarType::Byte, 0);
    return {p, (size_t)THPVariable_Unpack(o).numel()};
}

int32_t element_type(PyObject* o, const char* name, ScalarType* type) {
    if (THPVariable_Check(o)) {
        *type = THPVariable_Unpack(o).scalar_type();
        if (*type == ScalarType::BFloat16) return GS_TYPE_BF16;
        if (*type == ScalarType::Float) return GS_TYPE_F32;
    }
    throw ValueError(text(name, ": expected a float32 or bfloat16 tensor"));
}

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw TypeError("");
    return (float)v;
}

// what an object is as a condition; one that has no truth value raises
int32_t truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw TypeError("");
    return v;
}

// a tensor's size where the library takes 32 bits
int32_t small(int64_t n, const char* name) {
    if (n > INT32_MAX) throw ValueError(text(name, ": a dimension of ", n, " is too large"));
    return (int32_t)n;
}

// None: torch's current stream; an address; or an object with cuda_stream
void* stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* v = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!v) throw TypeError("");
    void* p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw TypeError("");
    return p;
}

// The library's call, without the interpreter's lock: a launch may wait for room in the queue.
template <typename F, typename... A>
gs_status unlocked(F* call, const A&... args) {
    PyThreadState* thread = PyEval_SaveThread();
    const gs_status st = call(args...);
    PyEval_RestoreThread(thread);
    return st;
}

struct Norm {
    int64_t tokens;
    int32_t hq, hk, dim;
    ScalarType type;
    gs_head_norm norm;
    gs_heads q, k;
    const float *qw, *kw, *table;
    const int32_t* positions;
    const Tensor *tq, *tk;
};

// q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved
Norm norm_of(PyObject* const* a, PyObject* eps, PyObject* interleaved) {
    Norm r{};
    r.norm.type = element_type(a[0], "q", &r.type);
    r.q = heads(a[0], "q", r.type);
    r.k = heads(a[1], "k", r.type);
    r.tq = &THPVariable_Unpack(a[0]);
    r.tk = &THPVariable_Unpack(a[1]);
    r.tokens = r.tq->size(0);
    r.hq = small(r.tq->size(1), "q");
    r.hk = small(r.tk->size(1), "k");
    r.dim = small(r.tq->size(2), "q");
    if (r.tk->size(0) != r.tokens || r.tk->size(2) != r.dim)
        throw ValueError(text("k: expected ", r.tokens, " tokens of ", r.dim,
                              " values a head, got ", r.tk->sizes()));
    r.qw = weights(a[2], "q_weight", r.dim);
    r.kw = weights(a[3], "k_weight", r.dim);
    if (a[4] != Py_None) {
        if (!THPVariable_Check(a[4]) || THPVariable_Unpack(a[4]).dim() != 2)
            throw ValueError("cos_sin: expected a [rows, rot] tensor");
        r.table = static_cast<float*>(flat(a[4], "cos_sin", ScalarType::Float, 0));
        r.norm.table_rows = THPVariable_Unpack(a[4]).size(0);
        r.norm.rot = small(THPVariable_Unpack(a[4]).size(1), "cos_sin");
    }
    r.positions = static_cast<int32_t*>(flat(a[5], "positions", ScalarType::Int, r.tokens, true));
    r.norm.eps = number(eps);
    r.norm.interleaved = truth(interleaved);
    return r;
}

gs_status qk_norm_rope(PyObject* const* a) {
    const Norm n = norm_of(a, a[8], a[9]);
    const gs_heads qo = heads(a[6], "q_out", n.type, n.tq), ko = heads(a[7], "k_out", n.type, n.tk);
    return unlocked(gs_qk_norm_rope, n.tokens, n.hq, n.hk, n.dim, &n.norm, &n.q, &n.k, n.qw, n.kw,
                    n.table, n.positions, &qo, &ko, stream_of(a[10]));
}

gs_status qk_norm_rope_bwd(PyObject* const* a) {
    const Norm n = norm_of(a, a[13], a[14]);
    const gs_heads yq = heads(a[6], "dq_out", n.type, n.tq), yk = heads(a[7], "dk_out", n.type, n.tk),
                   dq = heads(a[8], "dq", n.type, n.tq), dk = heads(a[9], "dk", n.type, n.tk);
    float *dqw = weights(a[10], "dq_weight", n.dim), *dkw = weights(a[11], "dk_weight", n.dim);
    const Bytes ws = workspace(a[12]);
    return unlocked(gs_qk_norm_rope_bwd, n.tokens, n.hq, n.hk, n.dim, &n.norm, &n.q, &n.k, n.qw, n.kw,
                    n.table, n.positions, &yq, &yk, &dq, &dk, dqw, dkw, ws.p, ws.n,
                    stream_of(a[15]));
}

struct Attention {
    gs_attention_shape shape;
    gs_heads q, k, v;
    const int32_t *cu_q, *cu_k;
    const Tensor *tq, *tk;
};

Attention attention_of(PyObject* q, PyObject* k, PyObject* v, PyObject* cu_q, PyObject* cu_k,
                       PyObject* causal, PyObject* scale) {
    const ScalarType bf = ScalarType::BFloat16;
    Attention r{};
    r.q = heads(q, "q", bf);
    r.k = heads(k, "k", bf);
    r.tq = &THPVariable_Unpack(q);
    r.tk = &THPVariable_Unpack(k);
    r.v = heads(v, "v", bf, r.tk);
    const int64_t dim = r.tq->size(2);
    if (r.tk->size(2) != dim)
        throw ValueError(text("k: expected ", dim, " values a head, got ", r.tk->sizes()));
    r.shape.batch = 1;
    if (cu_q != Py_None || cu_k != Py_None) {
        if (cu_q == Py_None || cu_k == Py_None)
            throw ValueError("cu_q and cu_k: give both or neither");
        r.cu_q = static_cast<int32_t*>(flat(cu_q, "cu_q", ScalarType::Int, 2));
        const int64_t n = THPVariable_Unpack(cu_q).numel();
        r.cu_k = static_cast<int32_t*>(flat(cu_k, "cu_k", ScalarType::Int, n));
        if (THPVariable_Unpack(cu_k).numel() != n)
            throw ValueError("cu_q and cu_k: expected batch + 1 offsets each");
        r.shape.batch = small(n - 1, "cu_q");
    }
    r.shape.tokens_q = r.tq->size(0);
    r.shape.tokens_k = r.tk->size(0);
    r.shape.heads_q = small(r.tq->size(1), "q");
    r.shape.heads_k = small(r.tk->size(1), "k");
    r.shape.head_dim = small(dim, "q");
    r.shape.causal = truth(causal);
    r.shape.scale = scale == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : number(scale);
    return r;
}

gs_status attention_fwd(PyObject* const* a) {
    const Attention t = attention_of(a[0], a[1], a[2], a[6], a[7], a[8], a[9]);
    const gs_heads out = heads(a[3], "out", ScalarType::BFloat16, t.tq);
    float* lse = static_cast<float*>(
        flat(a[4], "lse", ScalarType::Float, t.shape.tokens_q * t.shape.heads_q));
    const Bytes ws = workspace(a[5]);
    return unlocked(gs_attention_fwd, &t.shape, &t.q, &t.k, &t.v, t.cu_q, t.cu_k, &out, lse, ws.p,
                    ws.n, stream_of(a[10]));
}

gs_status attention_bwd(PyObject* const* a) {
    const ScalarType bf = ScalarType::BFloat16;
    const Attention t = attention_of(a[0], a[1], a[2], a[10], a[11], a[12], a[13]);
    const gs_heads out = heads(a[3], "out", bf, t.tq), dout = heads(a[5], "dout", bf, t.tq),
                   dq = heads(a[6], "dq", bf, t.tq), dk = heads(a[7], "dk", bf, t.tk),
                   dv = heads(a[8], "dv", bf, t.tk);
    const float* lse = static_cast<float*>(
        flat(a[4], "lse", ScalarType::Float, t.shape.tokens_q * t.shape.heads_q));
    const Bytes ws = workspace(a[9]);
    return unlocked(gs_attention_bwd, &t.shape, &t.q, &t.k, &t.v, t.cu_q, t.cu_k, &out, lse, &dout,
                    &dq, &dk, &dv, ws.p, ws.n, stream_of(a[14]));
}

const int64_t* rng_of(PyObject* o) {
    return static_cast<int64_t*>(flat(o, "rng", ScalarType::Long, 2));
}

gs_status dropout_add(PyObject* const* a) {
    ScalarType type;
    const int32_t kind = element_type(a[0], "x", &type);
    const void* x = flat(a[0], "x", type, 0);
    const Tensor& t = THPVariable_Unpack(a[0]);
    const int64_t n = t.numel();
    const void* residual = alike(a[1], "residual", t, true);
    void* out = alike(a[2], "out", t);
    return unlocked(gs_dropout_add, n, kind, x, residual, out, rng_of(a[3]), number(a[4]),
                    stream_of(a[5]));
}

gs_status dropout_add_bwd(PyObject* const* a) {
    ScalarType type;
    const int32_t kind = element_type(a[0], "dout", &type);
    const void* dout = flat(a[0], "dout", type, 0);
    const Tensor& t = THPVariable_Unpack(a[0]);
    const int64_t n = t.numel();
    void* dx = alike(a[1], "dx", t);
    return unlocked(gs_dropout_add_bwd, n, kind, dout, dx, rng_of(a[2]), number(a[3]), stream_of(a[4]));
}

// a call with its number of arguments; no C++ exception leaves it
template <gs_status (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)kCall(args));
    } catch (const TypeError& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const ValueError& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <gs_status (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kCall, kArgs>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<qk_norm_rope, 11>("qk_norm_rope"),
                         method<qk_norm_rope_bwd, 16>("qk_norm_rope_bwd"),
                         method<attention_fwd, 11>("attention_fwd"),
                         method<attention_bwd, 15>("attention_bwd"),
                         method<dropout_add, 6>("dropout_add"),
                         method<dropout_add_bwd, 5>("dropout_add_bwd"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gs_token_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gs_token_binding() { return PyModule_Create(&module); }
