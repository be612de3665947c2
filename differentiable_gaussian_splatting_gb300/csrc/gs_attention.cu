// gs_attention.cu -- softmax attention over ragged batches with shared key heads,
// and its gradient by recomputing the probabilities.
//
// One warp per row: the forward walks a query's keys with a running maximum and
// sum; the gradient takes one warp per query for dq and one per key for dk and dv,
// so that no two warps add to the same value.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gs_attention.cuh"
#include "gs_device.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {

namespace {

__device__ unsigned int g_gave_up;

constexpr int kAtThreads = 128;
constexpr int kPer = 4;  // values of a head per lane: head_dim <= 128

struct AtParams {
    int64_t tq, tk;
    int batch, hq, hk, dim, causal;
    float scale;
    HeadView q, k, v, o, dout, dq, dk, dv;
    const float* lse;
    float* delta;
    const int32_t *cu_q, *cu_k;
};

struct Span {
    int64_t q0, q1, k0, k1;
};

// the bounds of sequence b, kept inside the arrays
__device__ Span span_of(const AtParams& p, int b) {
    Span s;
    s.q0 = p.cu_q ? min64(max64(p.cu_q[b], 0), p.tq) : 0;
    s.q1 = p.cu_q ? min64(max64(p.cu_q[b + 1], s.q0), p.tq) : p.tq;
    s.k0 = p.cu_k ? min64(max64(p.cu_k[b], 0), p.tk) : 0;
    s.k1 = p.cu_k ? min64(max64(p.cu_k[b + 1], s.k0), p.tk) : p.tk;
    return s;
}

// the sequence that holds token t by its offsets (-1: none)
__device__ int sequence_of(const int32_t* cu, int batch, int64_t t) {
    if (!cu) return 0;
    for (int b = 0; b < batch; ++b)
        if (t >= cu[b] && t < cu[b + 1]) return b;
    return -1;
}

__device__ void load_row(float (&v)[kPer], const __nv_bfloat16* p, int dim) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < dim ? __bfloat162float(p[e]) : 0.f;
    }
}

__device__ void store_row(__nv_bfloat16* p, const float (&v)[kPer], int dim, float f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i < dim) p[lane + 32 * i] = __float2bfloat16_rn(v[i] * f);
}

__device__ float warp_dot(const float (&a)[kPer], const float (&b)[kPer]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

__global__ void __launch_bounds__(kAtThreads) attention_bwd_dq_simple(AtParams p) {
    grid_dep_sync();
    const int64_t w = ((int64_t)blockIdx.x * kAtThreads + threadIdx.x) >> 5;
    if (w >= p.tq * p.hq) return;
    const int64_t t = w / p.hq;
    const int h = (int)(w % p.hq), kh = h / (p.hq / p.hk);
    const int b = sequence_of(p.cu_q, p.batch, t);
    if (b < 0) return;
    const Span s = span_of(p, b);
    int64_t end = s.k1;
    if (p.causal) end = min64(s.k1, t - s.q0 + 1 + (s.k1 - s.k0) - (s.q1 - s.q0) + s.k0);
    float q[kPer], k[kPer], v[kPer], d[kPer], o[kPer], acc[kPer] = {};
    load_row(q, p.q.row(t, h), p.dim);
    load_row(o, p.o.row(t, h), p.dim);
    load_row(d, p.dout.row(t, h), p.dim);
    const float delta = warp_dot(o, d), lse = p.lse[h * p.tq + t];
    if ((threadIdx.x & 31) == 0) p.delta[h * p.tq + t] = delta;
    for (int64_t j = s.k0; j < end; ++j) {
        load_row(k, p.k.row(j, kh), p.dim);
        load_row(v, p.v.row(j, kh), p.dim);
        const float e = __expf(warp_dot(q, k) * p.scale - lse);
        const float ds = e * (warp_dot(d, v) - delta);
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = fmaf(ds, k[i], acc[i]);
    }
    store_row(p.dq.row(t, h), acc, p.dim, p.scale);
}

__global__ void __launch_bounds__(kAtThreads) attention_bwd_dkv_simple(AtParams p) {
    grid_dep_sync();
    const int64_t w = ((int64_t)blockIdx.x * kAtThreads + threadIdx.x) >> 5;
    if (w >= p.tk * p.hk) return;
    const int64_t j = w / p.hk;
    const int kh = (int)(w % p.hk), group = p.hq / p.hk;
    const int b = sequence_of(p.cu_k, p.batch, j);
    if (b < 0) return;
    const Span s = span_of(p, b);
    int64_t first = s.q0;
    if (p.causal) first = max64(s.q0, j - s.k0 - (s.k1 - s.k0) + (s.q1 - s.q0) + s.q0);
    float k[kPer], v[kPer], q[kPer], d[kPer], dk[kPer] = {}, dv[kPer] = {};
    load_row(k, p.k.row(j, kh), p.dim);
    load_row(v, p.v.row(j, kh), p.dim);
    for (int h = kh * group; h < (kh + 1) * group; ++h)
        for (int64_t t = first; t < s.q1; ++t) {
            load_row(q, p.q.row(t, h), p.dim);
            load_row(d, p.dout.row(t, h), p.dim);
            const float e = __expf(warp_dot(q, k) * p.scale - p.lse[h * p.tq + t]);
            const float ds = e * (warp_dot(d, v) - p.delta[h * p.tq + t]);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                dk[i] = fmaf(ds, q[i], dk[i]);
                dv[i] = fmaf(e, d[i], dv[i]);
            }
        }
    store_row(p.dk.row(j, kh), dk, p.dim, p.scale);
    store_row(p.dv.row(j, kh), dv, p.dim, 1.f);
}

HeadView view(const gs_heads& h) {
    return {static_cast<__nv_bfloat16*>(h.data), h.token_stride, h.head_stride};
}

AtParams params(const gs_attention_shape& s, const gs_heads& q, const gs_heads& k,
                const gs_heads& v, const gs_heads& o, const int32_t* cu_q, const int32_t* cu_k) {
    AtParams p{};
    p.tq = s.tokens_q;
    p.tk = s.tokens_k;
    p.batch = s.batch;
    p.hq = s.heads_q;
    p.hk = s.heads_k;
    p.dim = s.head_dim;
    p.causal = s.causal;
    p.scale = s.scale;
    p.q = view(q);
    p.k = view(k);
    p.v = view(v);
    p.o = view(o);
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    return p;
}

dim3 warps(int64_t n) { return dim3((unsigned)((n * 32 + kAtThreads - 1) / kAtThreads)); }

}  // namespace

size_t attention_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads_q,
                                 int heads_k, int head_dim) {
    (void)tokens_k, (void)batch, (void)heads_k, (void)head_dim;
    return ((size_t)tokens_q * heads_q * sizeof(float) + 255) / 256 * 256 + 256;
}

cudaError_t gave_up_word(unsigned int** word) {
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_gave_up);
    *word = static_cast<unsigned int*>(p);
    return e;
}

cudaError_t head_map(CUtensorMap* map, const void* data, int64_t ts, int64_t hs, int64_t tokens,
                     int heads, int dim, bool* swapped) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    // the driver's function, looked up once (a function's address does not change)
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return cudaErrorNotSupported;
    *swapped = ts < hs;
    const cuuint64_t size[3] = {(cuuint64_t)dim, (cuuint64_t)(*swapped ? tokens : heads),
                                (cuuint64_t)(*swapped ? heads : tokens)};
    const cuuint64_t stride[2] = {(cuuint64_t)(*swapped ? ts : hs) * 2,
                                  (cuuint64_t)(*swapped ? hs : ts) * 2};
    const cuuint32_t box[3] = {kBlockCols, *swapped ? kTileRows : 1u, *swapped ? 1u : kTileRows};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(data),
                              size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_attention_bwd(const gs_attention_shape& s, const gs_heads& q, const gs_heads& k,
                                 const gs_heads& v, const gs_heads& out, const float* lse,
                                 const gs_heads& dout, const gs_heads& dq, const gs_heads& dk,
                                 const gs_heads& dv, const int32_t* cu_q, const int32_t* cu_k,
                                 void* ws, cudaStream_t st) {
    AtParams p = params(s, q, k, v, out, cu_q, cu_k);
    p.lse = lse;
    p.delta = static_cast<float*>(ws);
    p.dout = view(dout);
    p.dq = view(dq);
    p.dk = view(dk);
    p.dv = view(dv);
    if (s.tokens_q > 0) {
        const cudaError_t e =
            launch(attention_bwd_dq_simple, warps(p.tq * p.hq), dim3(kAtThreads), 0, st, p);
        if (e != cudaSuccess) return e;
    }
    if (s.tokens_k == 0) return cudaSuccess;
    return launch(attention_bwd_dkv_simple, warps(p.tk * p.hk), dim3(kAtThreads), 0, st, p);
}

}  // namespace gs
