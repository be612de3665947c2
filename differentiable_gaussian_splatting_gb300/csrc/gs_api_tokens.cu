// gs_api_tokens.cu -- the extern "C" entry points of the token operators (see
// include/gs.h): argument checks on the host, before anything is enqueued.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gs_internal.h"
#include "gs_tokens.h"

using namespace gs;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;  // row and tile numbers stay in 32 bits
constexpr int64_t kMaxStride = int64_t(1) << 38;  // elements
constexpr int32_t kMaxHeads = 1024;
constexpr int32_t kMaxBatch = 1 << 20;
constexpr int32_t kMaxNormDim = 256, kMaxAttentionDim = 128;

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

gs_status gs_attention_fwd(const gs_attention_shape* shape, const gs_heads* q, const gs_heads* k,
                           const gs_heads* v, const int32_t* cu_q, const int32_t* cu_k,
                           const gs_heads* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (!shape_ok(shape)) return GS_ERR_INVALID_ARG;
    const gs_attention_shape& s = *shape;
    if (s.tokens_q == 0) return GS_OK;
    if (!offsets_ok(s, cu_q, cu_k) || !lse || !aligned16(lse) || !workspace ||
        !aligned16(workspace) || !heads_ok(q, s.tokens_q, s.heads_q, s.head_dim, 2) ||
        !heads_ok(k, s.tokens_k, s.heads_k, s.head_dim, 2) ||
        !heads_ok(v, s.tokens_k, s.heads_k, s.head_dim, 2) ||
        !heads_ok(out, s.tokens_q, s.heads_q, s.head_dim, 2))
        return GS_ERR_INVALID_ARG;
    if (workspace_bytes < gs_attention_workspace_bytes(shape)) return GS_ERR_WORKSPACE;
    return status_of(launch_attention_fwd(
        s, normal(q, s.tokens_q, s.heads_q, s.head_dim),
        normal(k, s.tokens_k, s.heads_k, s.head_dim), normal(v, s.tokens_k, s.heads_k, s.head_dim),
        normal(out, s.tokens_q, s.heads_q, s.head_dim), lse, cu_q, cu_k, workspace,
        (cudaStream_t)stream));
}

gs_status gs_attention_bwd(const gs_attention_shape* shape, const gs_heads* q, const gs_heads* k,
                           const gs_heads* v, const int32_t* cu_q, const int32_t* cu_k,
                           const gs_heads* out, const float* lse, const gs_heads* dout,
                           const gs_heads* dq, const gs_heads* dk, const gs_heads* dv,
                           void* workspace, size_t workspace_bytes, void* stream) {
    if (!shape_ok(shape)) return GS_ERR_INVALID_ARG;
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
    if (workspace_bytes < gs_attention_workspace_bytes(shape)) return GS_ERR_WORKSPACE;
    const auto nq = [&](const gs_heads* h) {
        return normal(h, s.tokens_q, s.heads_q, s.head_dim);
    };
    const auto nk = [&](const gs_heads* h) {
        return normal(h, s.tokens_k, s.heads_k, s.head_dim);
    };
    return status_of(launch_attention_bwd(s, nq(q), nk(k), nk(v), nq(out), lse, nq(dout), nq(dq),
                                          nk(dk), nk(dv), cu_q, cu_k, workspace,
                                          (cudaStream_t)stream));
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

}  // extern "C"
