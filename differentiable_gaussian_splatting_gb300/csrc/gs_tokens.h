// gs_tokens.h -- launch declarations of the token operators (head norms with rotation,
// attention, dropout-add, residual norms, gradient clipping), shared by their translation
// units and the entry points in gs_api_tokens.cu.  Not part of the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/gs.h"

namespace gs {

// ---- head norms and rotation (gs_headnorm.cu) --------------------------------
struct HeadNormArgs {
    int64_t tokens;
    int hq, hk, dim, rot;
    int64_t table_rows;
    float eps;
    bool bf16, interleaved;
    const float *qw, *kw;        // [dim] or null
    const float* cos_sin;        // [table_rows][rot]
    const int32_t* positions;    // [tokens] or null
};
cudaError_t launch_headnorm(const HeadNormArgs& a, const gs_heads& q, const gs_heads& k,
                            const gs_heads& q_out, const gs_heads& k_out, cudaStream_t st);
size_t headnorm_workspace_bytes(int64_t tokens, int dim);
cudaError_t launch_headnorm_bwd(const HeadNormArgs& a, const gs_heads& q, const gs_heads& k,
                                const gs_heads& dq_out, const gs_heads& dk_out,
                                const gs_heads& dq, const gs_heads& dk, float* dqw, float* dkw,
                                void* ws, cudaStream_t st);

// ---- dropout-add (gs_dropout.cu) ------------------------------------------------
cudaError_t launch_dropout_add(int64_t n, bool bf16, const void* x, const void* residual,
                               void* out, const int64_t* rng, uint32_t dropped, cudaStream_t st);

// ---- attention (gs_attention.cu) --------------------------------------------------
size_t attention_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads_q,
                                 int heads_k, int head_dim);
size_t attention_fwd_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads,
                                     int head_dim);
cudaError_t launch_attention_fwd(const gs_attention_shape& s, const gs_heads& q, const gs_heads& k,
                                 const gs_heads& v, const gs_heads& out, float* lse,
                                 const int32_t* cu_q, const int32_t* cu_k, void* ws,
                                 cudaStream_t st);
size_t attention_bwd_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads_q,
                                     int heads_k, int head_dim);
cudaError_t launch_attention_bwd(const gs_attention_shape& s, const gs_heads& q, const gs_heads& k,
                                 const gs_heads& v, const gs_heads& out, const float* lse,
                                 const gs_heads& dout, const gs_heads& dq, const gs_heads& dk,
                                 const gs_heads& dv, const int32_t* cu_q, const int32_t* cu_k,
                                 const gs_window* window, void* ws, cudaStream_t st);
// the same over a window (window null in the gradient above: none)
size_t attention_window_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads_q,
                                        int heads_k, int head_dim, const gs_window& window);
size_t attention_window_fwd_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads,
                                            int head_dim, const gs_window& window);
size_t attention_window_bwd_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch,
                                            int heads_q, int heads_k, int head_dim,
                                            const gs_window& window);
bool few_queries(const gs_attention_shape& s);
cudaError_t launch_attention_tokens(const gs_attention_shape& s, const gs_window& window,
                                    const gs_heads& q, const gs_heads& k, const gs_heads& v,
                                    const gs_heads& out, float* lse, const int32_t* cu_q,
                                    const int32_t* cu_k, cudaStream_t st);
cudaError_t launch_attention_window_fwd(const gs_attention_shape& s, const gs_window& window,
                                        const gs_heads& q, const gs_heads& k, const gs_heads& v,
                                        const gs_heads& out, float* lse, const int32_t* cu_q,
                                        const int32_t* cu_k, void* ws, cudaStream_t st);

// ---- norms around a block with its gate and residual (gs_residual_norm.cu) ----------
struct ResidualNormArgs {
    int64_t tokens;
    int width, batch;
    bool bf16;
    int pre, post;  // GS_NORM_*
    float alpha, beta, eps;
    gs_norm_params w;
    const int32_t* cu;
};
cudaError_t launch_residual_norm(const ResidualNormArgs& a, const gs_rows& x, const gs_rows& y,
                                 const gs_rows& r, const gs_rows& h, cudaStream_t st);
size_t residual_norm_workspace_bytes(int width);
cudaError_t launch_residual_norm_bwd(const ResidualNormArgs& a, const gs_rows& x, const gs_rows& y,
                                     const gs_rows& dr, const gs_rows& dh, const gs_rows& dx,
                                     const gs_rows& dy, const gs_norm_grads& g, void* ws,
                                     cudaStream_t st);

// ---- gradient norm and clipping (gs_clip.cu) ------------------------------------------
size_t clip_workspace_bytes(int count);
cudaError_t launch_clip(int count, const gs_array* in, const gs_array* out, double max_norm,
                        float* norm, void* ws, cudaStream_t st);

// whether a wait of an attention kernel has given up since this thread's last call (waits for st)
cudaError_t attention_gave_up(cudaStream_t st, bool* gave_up);

}  // namespace gs
