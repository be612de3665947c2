// token_binding.cpp -- the Python binding of the token operators: checks torch tensors and
// passes plain pointers to the calls of include/gs.h.  What the package's Python code does
// for the other calls through ctypes is done here in C++, because these are called many
// times a training step on few tokens: on the GB300's Grace a call's host time is 3 to 4 us
// (6 for attention's gradient with its two launches) instead of 6 to 23.  Errors are those of
// the Python code: TypeError and ValueError for tensors; the status of the call is returned.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <exception>
#include <sstream>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/gs.h"

// The calls that came after the first ones are looked for weakly: the binding loads beside a
// library without them, which then says so.
#pragma weak gs_attention_window_fwd
#pragma weak gs_attention_window_bwd
#pragma weak gs_residual_norm
#pragma weak gs_residual_norm_bwd
#pragma weak gs_clip_grad_norm

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

// The device that this thread's call launches on (-1: there is none).  A kernel there that was given
// another device's memory would fault.
thread_local c10::DeviceIndex current_device = -1;

void look_up_device() {
    if (c10::cuda::GetDevice(&current_device) != cudaSuccess) current_device = -1;
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeError(text(name, ": expected a torch tensor"));
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) throw ValueError(text(name, ": must be a CUDA tensor"));
    if (current_device >= 0 && t.device().index() != current_device)
        throw ValueError(text(name, ": is on ", t.device(), ", the current device is cuda:",
                              (int)current_device));
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

// A number for which infinity has a meaning of its own: a finite one beyond fp32 does not become it.
float finite_or_infinite(PyObject* o) {
    const float f = number(o);
    return std::isinf(f) && !std::isinf(PyFloat_AsDouble(o)) ? std::copysign(FLT_MAX, f) : f;
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
    if (!call) throw std::runtime_error("libgs.so does not have this call: build it anew");
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

// left, right, sinks; windows wider than 32 bits hold are as wide as all keys
gs_window window_of(PyObject* const* a) {
    const auto whole = [](PyObject* o, const char* name) {
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) throw TypeError("");
        if (v < 0) throw ValueError(text(name, ": expected a number from 0 on, got ", v));
        return (int32_t)std::min<long long>(v, INT32_MAX);
    };
    return {whole(a[0], "left"), whole(a[1], "right"), whole(a[2], "sinks")};
}

gs_status attention_window_fwd(PyObject* const* a) {
    const Attention t = attention_of(a[0], a[1], a[2], a[9], a[10], a[11], a[12]);
    const gs_window w = window_of(a + 6);
    const gs_heads out = heads(a[3], "out", ScalarType::BFloat16, t.tq);
    float* lse = static_cast<float*>(
        flat(a[4], "lse", ScalarType::Float, t.shape.tokens_q * t.shape.heads_q));
    const Bytes ws = workspace(a[5]);
    return unlocked(gs_attention_window_fwd, &t.shape, &w, &t.q, &t.k, &t.v, t.cu_q, t.cu_k, &out, lse,
                    ws.p, ws.n, stream_of(a[13]));
}

gs_status attention_window_bwd(PyObject* const* a) {
    const ScalarType bf = ScalarType::BFloat16;
    const Attention t = attention_of(a[0], a[1], a[2], a[13], a[14], a[15], a[16]);
    const gs_window w = window_of(a + 10);
    const gs_heads out = heads(a[3], "out", bf, t.tq), dout = heads(a[5], "dout", bf, t.tq),
                   dq = heads(a[6], "dq", bf, t.tq), dk = heads(a[7], "dk", bf, t.tk),
                   dv = heads(a[8], "dv", bf, t.tk);
    const float* lse = static_cast<float*>(
        flat(a[4], "lse", ScalarType::Float, t.shape.tokens_q * t.shape.heads_q));
    const Bytes ws = workspace(a[9]);
    return unlocked(gs_attention_window_bwd, &t.shape, &w, &t.q, &t.k, &t.v, t.cu_q, t.cu_k, &out, lse,
                    &dout, &dq, &dk, &dv, ws.p, ws.n, stream_of(a[17]));
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

// [tokens][width], contiguous in its last dimension, of the shape of `like`; or none
gs_rows rows(PyObject* o, const char* name, ScalarType type, const Tensor* like) {
    if (o == Py_None) return {nullptr, 0};
    const Tensor& t = tensor(o, name);
    if (t.dim() != 2) throw ValueError(text(name, ": expected [tokens, width], got ", t.sizes()));
    if (like && t.sizes() != like->sizes())
        throw ValueError(text(name, ": expected shape ", like->sizes(), ", got ", t.sizes()));
    want_type(t, name, type);
    if (t.stride(1) != 1 && t.size(1) > 1 && t.numel() > 0)
        throw ValueError(text(name, ": the last dimension must be contiguous"));
    return {address(t), t.stride(0)};
}

// n values of fp32, or null for None
float* vector(PyObject* o, const char* name, int64_t n) {
    void* p = flat(o, name, ScalarType::Float, n, true);
    if (o != Py_None && THPVariable_Unpack(o).numel() != n)
        throw ValueError(text(name, ": expected ", n, " values, got ", THPVariable_Unpack(o).sizes()));
    return static_cast<float*>(p);
}

struct BlockNorm {
    int64_t tokens, width;
    ScalarType type;
    gs_block_norm norm;
    gs_rows x, y;
    gs_norm_params w;
    const int32_t* cu;
    const Tensor* tx;
};

// a: pre_weight, pre_bias, post_weight, post_bias, gate, cu, pre, post, alpha, beta, eps
BlockNorm block_norm_of(PyObject* x, PyObject* y, PyObject* const* a) {
    BlockNorm r{};
    r.norm.type = element_type(x, "x", &r.type);
    r.x = rows(x, "x", r.type, nullptr);
    r.tx = &THPVariable_Unpack(x);
    r.y = rows(y, "y", r.type, r.tx);
    r.tokens = r.tx->size(0);
    r.width = small(r.tx->size(1), "x");
    r.norm.batch = 1;
    if (a[5] != Py_None) {
        r.cu = static_cast<int32_t*>(flat(a[5], "cu", ScalarType::Int, 2));
        r.norm.batch = small(THPVariable_Unpack(a[5]).numel() - 1, "cu");
    }
    r.w = {vector(a[0], "pre_weight", r.width), vector(a[1], "pre_bias", r.width),
           vector(a[2], "post_weight", r.width), vector(a[3], "post_bias", r.width),
           vector(a[4], "gate", r.norm.batch * r.width)};
    if (a[5] != Py_None && a[4] == Py_None) throw ValueError("cu: the offsets of a gate, which is None");
    r.norm.pre = (int32_t)number(a[6]);
    r.norm.post = (int32_t)number(a[7]);
    r.norm.alpha = number(a[8]);
    r.norm.beta = number(a[9]);
    r.norm.eps = number(a[10]);
    return r;
}

gs_status residual_norm(PyObject* const* a) {
    const BlockNorm n = block_norm_of(a[0], a[1], a + 4);
    const gs_rows r = rows(a[2], "r_out", n.type, n.tx), h = rows(a[3], "h_out", n.type, n.tx);
    return unlocked(gs_residual_norm, n.tokens, (int32_t)n.width, &n.norm, &n.x, &n.y, &n.w, n.cu, &r,
                    &h, stream_of(a[15]));
}

gs_status residual_norm_bwd(PyObject* const* a) {
    const BlockNorm n = block_norm_of(a[0], a[1], a + 7);
    const gs_rows dr = rows(a[2], "dr_out", n.type, n.tx), dh = rows(a[3], "dh_out", n.type, n.tx),
                  dx = rows(a[4], "dx", n.type, n.tx), dy = rows(a[5], "dy", n.type, n.tx);
    const Bytes ws = workspace(a[6]);
    const gs_norm_grads g{vector(a[18], "dpre_weight", n.width), vector(a[19], "dpre_bias", n.width),
                          vector(a[20], "dpost_weight", n.width),
                          vector(a[21], "dpost_bias", n.width),
                          vector(a[22], "dgate", n.norm.batch * n.width)};
    return unlocked(gs_residual_norm_bwd, n.tokens, (int32_t)n.width, &n.norm, &n.x, &n.y, &n.w, n.cu,
                    &dr, &dh, &dx, &dy, &g, ws.p, ws.n, stream_of(a[23]));
}

// the tensors of a list or tuple, contiguous, float32 or bfloat16
std::vector<gs_array> arrays(PyObject* o, const char* name, const std::vector<gs_array>* like) {
    if (!PyList_Check(o) && !PyTuple_Check(o))
        throw TypeError(text(name, ": expected a list or tuple of tensors"));
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
    if (like && n != (Py_ssize_t)like->size())
        throw ValueError(text(name, ": expected ", like->size(), " tensors, got ", n));
    std::vector<gs_array> r((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const Tensor& t = tensor(PySequence_Fast_GET_ITEM(o, i), name);
        const ScalarType type = t.scalar_type();
        if (type != ScalarType::Float && type != ScalarType::BFloat16)
            throw ValueError(text(name, "[", i, "]: expected float32 or bfloat16, got ", type));
        if (!t.is_contiguous()) throw ValueError(text(name, "[", i, "]: must be contiguous"));
        r[i] = {address(t), t.numel(), type == ScalarType::BFloat16 ? GS_TYPE_BF16 : GS_TYPE_F32};
        if (like && (r[i].elements != (*like)[i].elements || r[i].type != (*like)[i].type))
            throw ValueError(text(name, "[", i, "]: expected ", (*like)[i].elements,
                                  " elements of its gradient's type, got ", t.sizes(), " of ", type));
    }
    return r;
}

gs_status clip_grad_norm(PyObject* const* a) {
    const std::vector<gs_array> g = arrays(a[0], "grads", nullptr);
    float* norm = static_cast<float*>(flat(a[2], "norm", ScalarType::Float, 1));
    const Bytes ws = workspace(a[3]);
    std::vector<gs_array> o;
    if (a[4] != Py_None) o = arrays(a[4], "outs", &g);
    return unlocked(gs_clip_grad_norm, small((int64_t)g.size(), "grads"), g.data(),
                    a[4] != Py_None ? o.data() : nullptr, finite_or_infinite(a[1]), norm, ws.p, ws.n,
                    stream_of(a[5]));
}

// a call with its number of arguments; no C++ exception leaves it
template <gs_status (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        look_up_device();
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
                         method<attention_window_fwd, 14>("attention_window_fwd"),
                         method<attention_window_bwd, 18>("attention_window_bwd"),
                         method<residual_norm, 16>("residual_norm"),
                         method<residual_norm_bwd, 24>("residual_norm_bwd"),
                         method<clip_grad_norm, 6>("clip_grad_norm"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gs_token_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gs_token_binding() { return PyModule_Create(&module); }
