// gs_api_tokens.cu -- the extern "C" entry points of the token operators (see
// include/gs.h): argument checks on the host, before anything is enqueued.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "gs_internal.h"
#include "gs_tokens.h"

using namespace gs;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;  // row and tile numbers stay in 32 bits
constexpr int64_t kMaxStride = int64_t(1) << 38;  // elements
constexpr int32_t kMaxHeads = 1024;
constexpr int32_t kMaxBatch = 1 << 20;
constexpr int32_t kMaxNormDim = 256, kMaxAttentionDim = 128;
constexpr int32_t kMaxSinks = 128;  // of one key tile
// Sequences times query heads of a call by tiles with a window.  Every sequence has places for its tiles,
// used or not, and a CTA's planner takes 0.8 us (forward) or 1.3 us (gradient, whose two kinds of blocks
// of keys follow each other) to find one empty: 0.6 s at most, while waits give up after two.
constexpr int64_t kMaxWindowPlaces = int64_t(1) << 25;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

gs_status status_of(cudaError_t e) { return e == cudaSuccess ? GS_OK : GS_ERR_CUDA; }

// A [tokens][heads][dim] array read by strides: rows of whole 16-byte words that do
// not overlap, one stride a multiple of the other (strides of dimensions of one
// element do not matter).  Nothing is read where tokens is 0.
bool heads_ok(const gs_heads* h, int64_t tokens, int heads, int dim, int size) {
    if (!h) return false;
    if (tokens == 0) return true;
    const int64_t words = 16 / size;
    if (!h->data || !aligned16(h->data)) return false;
    const int64_t ts = tokens > 1 ? h->token_stride : (int64_t)heads * dim;
    const int64_t hs = heads > 1 ? h->head_stride : dim;
    if (ts < dim || hs < dim || ts > kMaxStride || hs > kMaxStride || ts % words || hs % words)
        return false;
    if (tokens > 1 && heads > 1) {
        const int64_t lo = ts < hs ? ts : hs, hi = ts < hs ? hs : ts;
        const int64_t n = ts < hs ? tokens : heads;
        if (hi % lo || hi / lo < n) return false;
    }
    return true;
}

// with the strides of dimensions of one element set to something valid
gs_heads normal(const gs_heads* h, int64_t tokens, int heads, int dim) {
    gs_heads r = *h;
    if (heads <= 1) r.head_stride = dim;
    if (tokens <= 1) r.token_stride = (heads <= 1 ? dim : r.head_stride * heads);
    return r;
}

bool norm_ok(int64_t tokens, int32_t hq, int32_t hk, int32_t dim, const gs_head_norm* n) {
    if (!n || tokens < 0 || tokens > kMaxTokens || hq < 1 || hk < 1 || hq > kMaxHeads ||
        hk > kMaxHeads || dim < 8 || dim > kMaxNormDim || dim % 8)
        return false;
    if (!(n->eps > 0.f) || !std::isfinite(n->eps)) return false;
    if (n->rot < 0 || n->rot > dim || n->rot % 2) return false;
    if (n->rot > 0 && (n->table_rows < 1 || n->table_rows > kMaxTokens)) return false;
    return (n->type == GS_TYPE_F32 || n->type == GS_TYPE_BF16);
}

bool norm_pointers_ok(const gs_head_norm& n, const float* qw, const float* kw, const float* table,
                      const int32_t* positions, int64_t tokens) {
    if ((qw && !aligned16(qw)) || (kw && !aligned16(kw)) || (positions && !aligned16(positions)))
        return false;
    if (n.rot > 0 && (!table || !aligned16(table))) return false;
    // without positions token t takes row t of the table
    return n.rot == 0 || positions || tokens <= n.table_rows;
}

HeadNormArgs norm_args(int64_t tokens, int32_t hq, int32_t hk, int32_t dim, const gs_head_norm& n,
                       const float* qw, const float* kw, const float* table,
                       const int32_t* positions) {
    HeadNormArgs a{};
    a.tokens = tokens;
    a.hq = hq;
    a.hk = hk;
    a.dim = dim;
    a.rot = n.rot;
    a.table_rows = n.table_rows;
    a.eps = n.eps;
    a.bf16 = n.type == GS_TYPE_BF16;
    a.interleaved = n.interleaved != 0;
    a.qw = qw;
    a.kw = kw;
    a.cos_sin = table;
    a.positions = positions;
    return a;
}

bool shape_ok(const gs_attention_shape* s) {
    return s && s->tokens_q >= 0 && s->tokens_k >= 0 && s->tokens_q <= kMaxTokens &&
           s->tokens_k <= kMaxTokens && s->batch >= 1 && s->batch <= kMaxBatch && s->heads_q >= 1 &&
           s->heads_k >= 1 && s->heads_q <= kMaxHeads && s->heads_q % s->heads_k == 0 &&
           s->head_dim >= 8 && s->head_dim <= kMaxAttentionDim && s->head_dim % 8 == 0 &&
           std::isfinite(s->scale) && (s->causal == 0 || s->causal == 1);
}

bool offsets_ok(const gs_attention_shape& s, const int32_t* cu_q, const int32_t* cu_k) {
    if ((cu_q == nullptr) != (cu_k == nullptr)) return false;
    return cu_q ? aligned16(cu_q) && aligned16(cu_k) : s.batch == 1;
}

}  // namespace

extern "C" {

size_t gs_qk_norm_rope_workspace_bytes(int64_t tokens, int32_t heads_q, int32_t heads_k,
                                       int32_t head_dim) {
    if (tokens < 0 || heads_q < 1 || heads_k < 1 || heads_q > kMaxHeads || heads_k > kMaxHeads ||
        head_dim < 8 || head_dim > kMaxNormDim || head_dim % 8)
        return 0;
    return headnorm_workspace_bytes(tokens, head_dim);
}

gs_status gs_qk_norm_rope(int64_t tokens, int32_t heads_q, int32_t heads_k, int32_t head_dim,
                          const gs_head_norm* norm, const gs_heads* q, const gs_heads* k,
                          const float* q_weight, const float* k_weight, const float* cos_sin,
                          const int32_t* positions, const gs_heads* q_out, const gs_heads* k_out,
                          void* stream) {
    if (!norm_ok(tokens, heads_q, heads_k, head_dim, norm)) return GS_ERR_INVALID_ARG;
    if (tokens == 0) return GS_OK;
    const int size = norm->type == GS_TYPE_BF16 ? 2 : 4;
    if (!norm_pointers_ok(*norm, q_weight, k_weight, cos_sin, positions, tokens) ||
        !heads_ok(q, tokens, heads_q, head_dim, size) ||
        !heads_ok(k, tokens, heads_k, head_dim, size) ||
        !heads_ok(q_out, tokens, heads_q, head_dim, size) ||
        !heads_ok(k_out, tokens, heads_k, head_dim, size))
        return GS_ERR_INVALID_ARG;
    return status_of(launch_headnorm(
        norm_args(tokens, heads_q, heads_k, head_dim, *norm, q_weight, k_weight, cos_sin,
                  positions),
        normal(q, tokens, heads_q, head_dim), normal(k, tokens, heads_k, head_dim),
        normal(q_out, tokens, heads_q, head_dim), normal(k_out, tokens, heads_k, head_dim),
        (cudaStream_t)stream));
}

gs_status gs_qk_norm_rope_bwd(int64_t tokens, int32_t heads_q, int32_t heads_k, int32_t head_dim,
                              const gs_head_norm* norm, const gs_heads* q, const gs_heads* k,
                              const float* q_weight, const float* k_weight, const float* cos_sin,
                              const int32_t* positions, const gs_heads* dq_out,
                              const gs_heads* dk_out, const gs_heads* dq, const gs_heads* dk,
                              float* dq_weight, float* dk_weight, void* workspace,
                              size_t workspace_bytes, void* stream) {
    if (!norm_ok(tokens, heads_q, heads_k, head_dim, norm)) return GS_ERR_INVALID_ARG;
    const int size = norm->type == GS_TYPE_BF16 ? 2 : 4;
    if (!workspace || !aligned16(workspace) || (dq_weight && !aligned16(dq_weight)) ||
        (dk_weight && !aligned16(dk_weight)) ||
        !norm_pointers_ok(*norm, q_weight, k_weight, cos_sin, positions, tokens) ||
        !heads_ok(q, tokens, heads_q, head_dim, size) ||
        !heads_ok(k, tokens, heads_k, head_dim, size) ||
        !heads_ok(dq_out, tokens, heads_q, head_dim, size) ||
        !heads_ok(dk_out, tokens, heads_k, head_dim, size) ||
        !heads_ok(dq, tokens, heads_q, head_dim, size) ||
        !heads_ok(dk, tokens, heads_k, head_dim, size))
        return GS_ERR_INVALID_ARG;
    if (workspace_bytes < headnorm_workspace_bytes(tokens, head_dim)) return GS_ERR_WORKSPACE;
    return status_of(launch_headnorm_bwd(
        norm_args(tokens, heads_q, heads_k, head_dim, *norm, q_weight, k_weight, cos_sin,
                  positions),
        normal(q, tokens, heads_q, head_dim), normal(k, tokens, heads_k, head_dim),
        normal(dq_out, tokens, heads_q, head_dim), normal(dk_out, tokens, heads_k, head_dim),
        normal(dq, tokens, heads_q, head_dim), normal(dk, tokens, heads_k, head_dim), dq_weight,
        dk_weight, workspace, (cudaStream_t)stream));
}

size_t gs_attention_workspace_bytes(const gs_attention_shape* shape) {
    if (!shape_ok(shape)) return 0;
    return attention_workspace_bytes(shape->tokens_q, shape->tokens_k, shape->batch,
                                     shape->heads_q, shape->heads_k, shape->head_dim);
}

namespace {

// window: null without one
gs_status attention_fwd(const gs_attention_shape* shape, const gs_window* window, const gs_heads* q,
                        const gs_heads* k, const gs_heads* v, const int32_t* cu_q,
                        const int32_t* cu_k, const gs_heads* out, float* lse, void* workspace,
                        size_t workspace_bytes, size_t needed, void* stream) {
    const gs_attention_shape& s = *shape;
    if (s.tokens_q == 0) return GS_OK;
    if (!offsets_ok(s, cu_q, cu_k) || !lse || !aligned16(lse) || !workspace ||
        !aligned16(workspace) || !heads_ok(q, s.tokens_q, s.heads_q, s.head_dim, 2) ||
        !heads_ok(k, s.tokens_k, s.heads_k, s.head_dim, 2) ||
        !heads_ok(v, s.tokens_k, s.heads_k, s.head_dim, 2) ||
        !heads_ok(out, s.tokens_q, s.heads_q, s.head_dim, 2))
        return GS_ERR_INVALID_ARG;
    const bool few = window && few_queries(s);
    if (window && !few && (int64_t)s.batch * s.heads_q > kMaxWindowPlaces) return GS_ERR_INVALID_ARG;
    if (workspace_bytes < needed) return GS_ERR_WORKSPACE;
    const gs_heads nq = normal(q, s.tokens_q, s.heads_q, s.head_dim),
                   nk = normal(k, s.tokens_k, s.heads_k, s.head_dim),
                   nv = normal(v, s.tokens_k, s.heads_k, s.head_dim),
                   no = normal(out, s.tokens_q, s.heads_q, s.head_dim);
    if (few)
        return status_of(launch_attention_tokens(s, *window, nq, nk, nv, no, lse, cu_q, cu_k,
                                                 (cudaStream_t)stream));
    return status_of(window ? launch_attention_window_fwd(s, *window, nq, nk, nv, no, lse, cu_q, cu_k,
                                                          workspace, (cudaStream_t)stream)
                            : launch_attention_fwd(s, nq, nk, nv, no, lse, cu_q, cu_k, workspace,
                                                   (cudaStream_t)stream));
}

gs_status attention_bwd(const gs_attention_shape* shape, const gs_window* window, const gs_heads* q,
                        const gs_heads* k, const gs_heads* v, const int32_t* cu_q,
                        const int32_t* cu_k, const gs_heads* out, const float* lse,
                        const gs_heads* dout, const gs_heads* dq, const gs_heads* dk,
                        const gs_heads* dv, void* workspace, size_t workspace_bytes, size_t needed,
                        void* stream) {
    const gs_attention_shape& s = *shape;
    if (s.tokens_q == 0 && s.tokens_k == 0) return GS_OK;
    if (!offsets_ok(s, cu_q, cu_k) || (s.tokens_q > 0 && (!lse || !aligned16(lse))) || !workspace ||
        !aligned16(workspace))
        return GS_ERR_INVALID_ARG;
    const gs_heads* of_q[] = {q, out, dout, dq};
    const gs_heads* of_k[] = {k, v, dk, dv};
    for (const gs_heads* h : of_q)
        if (!heads_ok(h, s.tokens_q, s.heads_q, s.head_dim, 2)) return GS_ERR_INVALID_ARG;
    for (const gs_heads* h : of_k)
        if (!heads_ok(h, s.tokens_k, s.heads_k, s.head_dim, 2)) return GS_ERR_INVALID_ARG;
    if (window && (int64_t)s.batch * s.heads_q > kMaxWindowPlaces) return GS_ERR_INVALID_ARG;
    if (workspace_bytes < needed) return GS_ERR_WORKSPACE;
    const auto nq = [&](const gs_heads* h) {
        return normal(h, s.tokens_q, s.heads_q, s.head_dim);
    };
    const auto nk = [&](const gs_heads* h) {
        return normal(h, s.tokens_k, s.heads_k, s.head_dim);
    };
    return status_of(launch_attention_bwd(s, nq(q), nk(k), nk(v), nq(out), lse, nq(dout), nq(dq),
                                          nk(dk), nk(dv), cu_q, cu_k, window, workspace,
                                          (cudaStream_t)stream));
}

bool window_ok(const gs_window* w) {
    return w && w->left >= 0 && w->right >= 0 && w->sinks >= 0 && w->sinks <= kMaxSinks;
}

}  // namespace

gs_status gs_attention_fwd(const gs_attention_shape* shape, const gs_heads* q, const gs_heads* k,
                           const gs_heads* v, const int32_t* cu_q, const int32_t* cu_k,
                           const gs_heads* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (!shape_ok(shape)) return GS_ERR_INVALID_ARG;
    return attention_fwd(shape, nullptr, q, k, v, cu_q, cu_k, out, lse, workspace, workspace_bytes,
                         gs_attention_workspace_bytes(shape), stream);
}

gs_status gs_attention_bwd(const gs_attention_shape* shape, const gs_heads* q, const gs_heads* k,
                           const gs_heads* v, const int32_t* cu_q, const int32_t* cu_k,
                           const gs_heads* out, const float* lse, const gs_heads* dout,
                           const gs_heads* dq, const gs_heads* dk, const gs_heads* dv,
                           void* workspace, size_t workspace_bytes, void* stream) {
    if (!shape_ok(shape)) return GS_ERR_INVALID_ARG;
    return attention_bwd(shape, nullptr, q, k, v, cu_q, cu_k, out, lse, dout, dq, dk, dv, workspace,
                         workspace_bytes, gs_attention_workspace_bytes(shape), stream);
}

size_t gs_attention_window_workspace_bytes(const gs_attention_shape* shape,
                                           const gs_window* window) {
    if (!shape_ok(shape) || !window_ok(window)) return 0;
    return attention_window_workspace_bytes(shape->tokens_q, shape->tokens_k, shape->batch,
                                            shape->heads_q, shape->heads_k, shape->head_dim,
                                            *window);
}

gs_status gs_attention_window_fwd(const gs_attention_shape* shape, const gs_window* window,
                                  const gs_heads* q, const gs_heads* k, const gs_heads* v,
                                  const int32_t* cu_q, const int32_t* cu_k, const gs_heads* out,
                                  float* lse, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    if (!shape_ok(shape) || !window_ok(window)) return GS_ERR_INVALID_ARG;
    return attention_fwd(shape, window, q, k, v, cu_q, cu_k, out, lse, workspace, workspace_bytes,
                         gs_attention_window_workspace_bytes(shape, window), stream);
}

gs_status gs_attention_window_bwd(const gs_attention_shape* shape, const gs_window* window,
                                  const gs_heads* q, const gs_heads* k, const gs_heads* v,
                                  const int32_t* cu_q, const int32_t* cu_k, const gs_heads* out,
                                  const float* lse, const gs_heads* dout, const gs_heads* dq,
                                  const gs_heads* dk, const gs_heads* dv, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    if (!shape_ok(shape) || !window_ok(window)) return GS_ERR_INVALID_ARG;
    return attention_bwd(shape, window, q, k, v, cu_q, cu_k, out, lse, dout, dq, dk, dv, workspace,
                         workspace_bytes, gs_attention_window_workspace_bytes(shape, window),
                         stream);
}

gs_status gs_attention_status(void* stream) {
    bool gave_up = false;
    const cudaError_t e = attention_gave_up((cudaStream_t)stream, &gave_up);
    if (e != cudaSuccess) return GS_ERR_CUDA;
    return gave_up ? GS_ERR_TIMEOUT : GS_OK;
}

namespace {

bool dropout_ok(int64_t n, int32_t type, float p, uint32_t* dropped) {
    if (n < 0 || n > (int64_t(1) << 42) || (type != GS_TYPE_F32 && type != GS_TYPE_BF16))
        return false;
    if (!(p >= 0.f && p < 1.f)) return false;
    *dropped = (uint32_t)std::floor((double)p * 65536.0 + 0.5);
    return *dropped < 65536u;
}

}  // namespace

gs_status gs_dropout_add(int64_t n, int32_t type, const void* x, const void* residual, void* out,
                         const int64_t* rng, float p, void* stream) {
    uint32_t dropped = 0;
    if (!dropout_ok(n, type, p, &dropped)) return GS_ERR_INVALID_ARG;
    if (n == 0) return GS_OK;
    if (!x || !out || !rng || !aligned16(x) || !aligned16(out) || !aligned16(rng) ||
        (residual && !aligned16(residual)))
        return GS_ERR_INVALID_ARG;
    return status_of(launch_dropout_add(n, type == GS_TYPE_BF16, x, residual, out, rng, dropped,
                                        (cudaStream_t)stream));
}

gs_status gs_dropout_add_bwd(int64_t n, int32_t type, const void* dout, void* dx,
                             const int64_t* rng, float p, void* stream) {
    return gs_dropout_add(n, type, dout, nullptr, dx, rng, p, stream);
}

namespace {

constexpr int32_t kMaxWidth = 8192;
constexpr int64_t kMaxRowStride = int64_t(1) << 29;  // elements: bytes stay in 32 bits
constexpr int32_t kMaxArrays = 65536;

bool aligned(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size == 0; }

// a [tokens][width] array by rows that do not overlap; with `optional` it may be missing
bool rows_ok(const gs_rows* r, int64_t tokens, int width, int size, bool optional) {
    if (!r || !r->data) return optional || tokens == 0;
    return aligned(r->data, size) &&
           (tokens <= 1 || (r->row_stride >= width && r->row_stride <= kMaxRowStride));
}

// with a missing array's pointer null, and the stride of a single row set to something valid
gs_rows normal(const gs_rows* r, int64_t tokens, int width) {
    gs_rows n = r ? *r : gs_rows{nullptr, 0};
    if (tokens <= 1) n.row_stride = (width + 7) / 8 * 8;
    return n;
}

bool block_norm_ok(int64_t tokens, int32_t width, const gs_block_norm* n, const gs_rows* y,
                   const gs_norm_params* w, const int32_t* cu) {
    if (!n || !w || tokens < 0 || tokens > kMaxTokens || width < 1 || width > kMaxWidth) return false;
    if (n->type != GS_TYPE_F32 && n->type != GS_TYPE_BF16) return false;
    if (n->pre < GS_NORM_NONE || n->pre > GS_NORM_LAYER || n->post < GS_NORM_NONE ||
        n->post > GS_NORM_LAYER)
        return false;
    if (!std::isfinite(n->alpha) || !std::isfinite(n->beta) || !(n->eps > 0.f) ||
        !std::isfinite(n->eps))
        return false;
    if (n->pre == GS_NORM_NONE && (w->pre_weight || w->pre_bias)) return false;
    if (n->post == GS_NORM_NONE && (w->post_weight || w->post_bias)) return false;
    if ((!y || !y->data) && tokens > 0 && (n->post != GS_NORM_NONE || w->gate)) return false;
    if (n->batch < 1 || n->batch > kMaxBatch || (!cu && n->batch != 1) || (cu && !w->gate)) return false;
    for (const void* p : {(const void*)w->pre_weight, (const void*)w->pre_bias,
                          (const void*)w->post_weight, (const void*)w->post_bias,
                          (const void*)w->gate, (const void*)cu})
        if (!aligned16(p)) return false;
    return true;
}

// Whether no out of the arrays meets another, nor a gradient that is not its own.
bool outs_apart(int32_t count, const gs_array* grads, const gs_array* outs, gs_status* st) {
    struct Span {
        uintptr_t begin, end;
    };
    const auto span = [](const gs_array& a) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(a.data);
        return Span{at, at + (uintptr_t)a.elements * (a.type == GS_TYPE_BF16 ? 2 : 4)};
    };
    const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[(size_t)count + 1]);
    *st = spans ? GS_ERR_INVALID_ARG : GS_ERR_WORKSPACE;
    if (!spans) return false;
    int n = 0;
    for (int32_t i = 0; i < count; ++i)
        if (outs[i].elements > 0) spans[n++] = span(outs[i]);
    const auto before = [](const Span& a, const Span& b) { return a.begin < b.begin; };
    if (!std::is_sorted(&spans[0], &spans[n], before)) std::sort(&spans[0], &spans[n], before);
    for (int i = 1; i < n; ++i)
        if (spans[i].begin < spans[i - 1].end) return false;
    for (int32_t i = 0; i < count; ++i) {
        if (grads[i].data == outs[i].data || grads[i].elements == 0) continue;
        const Span g = span(grads[i]);  // the first out that ends behind its start
        const Span* o = std::upper_bound(&spans[0], &spans[n], g,
                                         [](const Span& a, const Span& b) { return a.begin < b.end; });
        if (o != &spans[n] && o->begin < g.end) return false;
    }
    return true;
}

ResidualNormArgs norm_args(int64_t tokens, int32_t width, const gs_block_norm& n,
                           const gs_norm_params& w, const int32_t* cu) {
    return {tokens,  width,  n.batch, n.type == GS_TYPE_BF16, n.pre, n.post,
            n.alpha, n.beta, n.eps,   w,                      cu};
}

}  // namespace

gs_status gs_residual_norm(int64_t tokens, int32_t width, const gs_block_norm* norm,
                           const gs_rows* x, const gs_rows* y, const gs_norm_params* params,
                           const int32_t* cu, const gs_rows* r_out, const gs_rows* h_out,
                           void* stream) {
    if (!block_norm_ok(tokens, width, norm, y, params, cu)) return GS_ERR_INVALID_ARG;
    if (tokens == 0) return GS_OK;
    const int size = norm->type == GS_TYPE_BF16 ? 2 : 4;
    const bool pre = norm->pre != GS_NORM_NONE;
    if (!rows_ok(x, tokens, width, size, false) || !rows_ok(y, tokens, width, size, true) ||
        !rows_ok(r_out, tokens, width, size, true) || !rows_ok(h_out, tokens, width, size, !pre) ||
        (!pre && h_out && h_out->data))
        return GS_ERR_INVALID_ARG;
    return status_of(launch_residual_norm(norm_args(tokens, width, *norm, *params, cu),
                                          normal(x, tokens, width), normal(y, tokens, width),
                                          normal(r_out, tokens, width),
                                          normal(h_out, tokens, width), (cudaStream_t)stream));
}

size_t gs_residual_norm_workspace_bytes(int64_t tokens, int32_t width, int32_t batch) {
    if (tokens < 0 || tokens > kMaxTokens || width < 1 || width > kMaxWidth || batch < 1 ||
        batch > kMaxBatch)
        return 0;
    return residual_norm_workspace_bytes(width);
}

gs_status gs_residual_norm_bwd(int64_t tokens, int32_t width, const gs_block_norm* norm,
                               const gs_rows* x, const gs_rows* y, const gs_norm_params* params,
                               const int32_t* cu, const gs_rows* dr_out, const gs_rows* dh_out,
                               const gs_rows* dx, const gs_rows* dy, const gs_norm_grads* grads,
                               void* workspace, size_t workspace_bytes, void* stream) {
    if (!block_norm_ok(tokens, width, norm, y, params, cu) || !grads) return GS_ERR_INVALID_ARG;
    const int size = norm->type == GS_TYPE_BF16 ? 2 : 4;
    const bool pre = norm->pre != GS_NORM_NONE, post = norm->post != GS_NORM_NONE;
    const bool of_y = y && y->data;
    if (!rows_ok(x, tokens, width, size, false) || !rows_ok(y, tokens, width, size, true) ||
        !rows_ok(dr_out, tokens, width, size, true) ||
        !rows_ok(dh_out, tokens, width, size, !pre) || (!pre && dh_out && dh_out->data) ||
        !rows_ok(dx, tokens, width, size, false) || !rows_ok(dy, tokens, width, size, !of_y) ||
        (tokens > 0 && !of_y && dy && dy->data))
        return GS_ERR_INVALID_ARG;
    if ((!pre && (grads->pre_weight || grads->pre_bias)) ||
        (!post && (grads->post_weight || grads->post_bias)) || (grads->gate && !params->gate))
        return GS_ERR_INVALID_ARG;
    for (const float* g : {grads->pre_weight, grads->pre_bias, grads->post_weight, grads->post_bias,
                           grads->gate})
        if (!aligned16(g)) return GS_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return GS_ERR_INVALID_ARG;
    if (workspace_bytes < residual_norm_workspace_bytes(width)) return GS_ERR_WORKSPACE;
    return status_of(launch_residual_norm_bwd(
        norm_args(tokens, width, *norm, *params, cu), normal(x, tokens, width),
        normal(y, tokens, width), normal(dr_out, tokens, width), normal(dh_out, tokens, width),
        normal(dx, tokens, width), normal(dy, tokens, width), *grads, workspace,
        (cudaStream_t)stream));
}

size_t gs_clip_grad_norm_workspace_bytes(int32_t count) {
    return count < 0 || count > kMaxArrays ? 0 : clip_workspace_bytes(count);
}

gs_status gs_clip_grad_norm(int32_t count, const gs_array* grads, const gs_array* outs,
                            float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                            void* stream) {
    if (count < 0 || count > kMaxArrays || (count > 0 && !grads) || !(max_norm >= 0.f) || !norm ||
        !aligned(norm, 4) || !workspace || !aligned16(workspace))
        return GS_ERR_INVALID_ARG;
    if (!outs) outs = grads;
    int64_t all = 0;
    for (int32_t i = 0; i < count; ++i) {
        const gs_array &g = grads[i], &o = outs[i];
        if ((g.type != GS_TYPE_F32 && g.type != GS_TYPE_BF16) || o.type != g.type ||
            g.elements < 0 || g.elements > (int64_t(1) << 40) || o.elements != g.elements)
            return GS_ERR_INVALID_ARG;
        const int size = g.type == GS_TYPE_BF16 ? 2 : 4;
        if (g.elements > 0 && (!g.data || !o.data || !aligned(g.data, size) || !aligned(o.data, size)))
            return GS_ERR_INVALID_ARG;
        all += g.elements;
    }
    if (all > (int64_t(1) << 42)) return GS_ERR_INVALID_ARG;
    gs_status st;
    if (!outs_apart(count, grads, outs, &st)) return st;
    if (workspace_bytes < clip_workspace_bytes(count)) return GS_ERR_WORKSPACE;
    return status_of(launch_clip(count, grads, outs, (double)max_norm, norm, workspace,
                                 (cudaStream_t)stream));
}

}  // extern "C"
