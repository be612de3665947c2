// gs_headnorm.cu -- RMS norm of every query and key head and the position
// rotation in one pass, and its gradient.
//
// A head's row x of D values becomes n = r w x with r = (mean x^2 + eps)^(-1/2);
// the first `rot` values of n are taken as rot/2 pairs (a, b) and turned by the
// token's angles: (a c - b s, b c + a s).  Both steps are linear in n, so a lane
// forms its outputs as r (A_j x_j + B_j x'_j), x'_j the other value of the pair,
// A_j = c w_j and B_j = -/+ s w'_j.  The gradient turns dy back by the same
// angles into g, and with s2 = sum x^2, t = sum_j w_j g_j x_j
//   dx_j = r (w_j g_j - x_j r^2 t / D),   dw_j = sum over rows of g_j x_j r,
// so one pass with two sums over the row serves it.
//
// Everything is bound by memory (about 14 operations for 6 bytes in bfloat16).
// A lane holds 8 neighbouring values (16 bytes of bfloat16), a row takes the next
// power of two of D / 8 lanes, and a warp keeps kRows rows of one token in flight.
// A warp stays on the queries or on the keys, so the norm weights are read once;
// the angles are read once for each token's rows in flight.  A pair whose other
// half lies in another lane is read again from global memory: the bytes are in
// L1, which costs less than moving eight values by shuffles.
//
// Sums are in 32 bits.  The weight gradients are summed per lane over a warp's
// tokens, per block in shared memory in warp order, and over blocks by a second
// kernel in block order: the same inputs give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gs_device.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {
namespace {

constexpr int kHnThreads = 256;
constexpr int kHnWarps = kHnThreads / 32;
constexpr int kHnMaxBlocks = 608;  // 4 blocks on each of 152 SMs
constexpr int kFinishCols = 32;

struct Rows {
    char* p;
    int64_t ts, hs;  // strides in bytes
};

struct HnParams {
    int64_t tokens, table_rows;
    int hq, hk, dim, rot;
    int chunks_q, chunks_k;  // kRows * (32 / lanes) heads each
    float eps;
    const float *qw, *kw, *cos_sin;
    const int32_t* positions;
    Rows q, k, yq, yk;    // inputs; outputs (forward) or the outputs' gradients (backward)
    Rows dq, dk;          // backward
    float* part;          // backward: [blocks][2][dim]
};

// eight values, raw
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
    __device__ void load(const char* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ void set(int k, const char* p) { (&(k < 4 ? a : b).x)[k & 3] = *reinterpret_cast<const float*>(p); }
    __device__ float get(int k) const {
        const float4& v = k < 4 ? a : b;
        return (k & 3) == 0 ? v.x : (k & 3) == 1 ? v.y : (k & 3) == 2 ? v.z : v.w;
    }
    __device__ static void store(char* p, const float (&v)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint32_t w[4];
    __device__ void load(const char* p) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    __device__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ void set(int k, const char* p) {
        const uint32_t h = *reinterpret_cast<const uint16_t*>(p);
        w[k >> 1] = (k & 1) ? (w[k >> 1] & 0xffffu) | (h << 16) : (w[k >> 1] & 0xffff0000u) | h;
    }
    __device__ float get(int k) const {
        return __uint_as_float((k & 1) ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
    }
    __device__ static void store(char* p, const float (&v)[8]) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
    }
};

// index of the value that value e of a row is paired with (itself: not rotated)
template <bool kInter>
__device__ __forceinline__ int partner(int e, int rot) {
    if (e >= rot) return e;
    if (kInter) return e ^ 1;
    const int h = rot >> 1;
    return e < h ? e + h : e - h;
}

// What a lane knows of its 8 columns: whether the partners of all of them are the
// 8 columns at `poff` (16-byte loads), or are to be read one by one.
struct Cols {
    int e0;        // first column
    bool in;       // e0 < dim
    bool any;      // some column is rotated
    bool vec;      // half-split partners are the 8 columns from poff
    int poff;
};

template <bool kInter>
__device__ __forceinline__ Cols columns(int lane, int dim, int rot) {
    Cols c;
    c.e0 = lane * 8;
    c.in = c.e0 < dim;
    c.any = c.in && c.e0 < rot;
    c.vec = !kInter && (rot >> 1) % 8 == 0;
    c.poff = c.any && !kInter ? partner<false>(c.e0, rot) : c.e0;
    return c;
}

// the other values of the pairs of 8 columns (0 where a column is not rotated)
template <typename T, bool kInter>
__device__ __forceinline__ void load_partner(Raw<T>& x, const char* row, const Cols& c, int rot) {
    if (c.vec) {
        x.load(row + c.poff * sizeof(T));
        return;
    }
    x.zero();
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c.e0 + k < rot) x.set(k, row + partner<kInter>(c.e0 + k, rot) * sizeof(T));
}

// cos and signed sin of the 8 columns of a token (1 and 0 where not rotated)
template <bool kInter>
__device__ __forceinline__ void load_angles(float (&co)[8], float (&si)[8], const Cols& c,
                                            const HnParams& p, int64_t pos, bool turned) {
#pragma unroll
    for (int k = 0; k < 8; ++k) co[k] = 1.f, si[k] = 0.f;
    if (!turned || !c.any) return;
    const int half = p.rot >> 1;
    if (pos >= p.table_rows) {  // not in the table: shows in the result
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c.e0 + k < p.rot) co[k] = si[k] = __int_as_float(0x7fc00000);
        return;
    }
    const float* row = p.cos_sin + pos * p.rot;
    if (c.vec) {
        const int i = c.e0 < half ? c.e0 : c.e0 - half;
        const float sign = c.e0 < half ? -1.f : 1.f;
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(row + i + k));
            const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + i + k));
            co[k] = a.x, co[k + 1] = a.y, co[k + 2] = a.z, co[k + 3] = a.w;
            si[k] = sign * b.x, si[k + 1] = sign * b.y, si[k + 2] = sign * b.z, si[k + 3] = sign * b.w;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int e = c.e0 + k;
        if (e >= p.rot) break;
        const bool first = kInter ? (e & 1) == 0 : e < half;
        const int i = kInter ? e >> 1 : (first ? e : e - half);
        co[k] = __ldg(row + i);
        si[k] = first ? -__ldg(row + half + i) : __ldg(row + half + i);
    }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A warp's place: queries or keys, its heads, its first token and its step.
struct Place {
    bool keys, active;
    int head0;
    int64_t token, step;
};

template <int kHeads>
__device__ __forceinline__ Place place(const HnParams& p) {
    const int chunks = p.chunks_q + p.chunks_k;
    const int warps = gridDim.x * kHnWarps, used = warps / chunks * chunks;
    const int w = blockIdx.x * kHnWarps + (threadIdx.x >> 5);
    Place s;
    s.active = w < used;
    const int c = w % chunks;
    s.keys = c >= p.chunks_q;
    s.head0 = (s.keys ? c - p.chunks_q : c) * kHeads;
    s.token = w / chunks;
    s.step = used / chunks;
    return s;
}

template <typename T, bool kInter, int kLanes, int kRows>
__global__ void __launch_bounds__(kHnThreads) headnorm_kernel(const HnParams p) {
    grid_dep_sync();
    constexpr int kSub = 32 / kLanes;
    const Place at = place<kSub * kRows>(p);
    if (!at.active) return;
    const int lane = threadIdx.x & (kLanes - 1), sub = (threadIdx.x & 31) / kLanes;
    const Cols c = columns<kInter>(lane, p.dim, p.rot);
    const Rows in = at.keys ? p.k : p.q, out = at.keys ? p.yk : p.yq;
    const int heads = at.keys ? p.hk : p.hq;
    const float* w = at.keys ? p.kw : p.qw;
    float wj[8], wo[8];  // weights of the columns and of their partners
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int e = c.e0 + k;
        wj[k] = w && c.in ? __ldg(w + e) : 1.f;
        wo[k] = w && c.in ? __ldg(w + partner<kInter>(e, p.rot)) : 1.f;
    }
    const float inv_dim = 1.f / (float)p.dim;
    for (int64_t t = at.token; t < p.tokens; t += at.step) {
        const int64_t pos = p.positions ? (int64_t)__ldg(p.positions + t) : t;
        const bool turned = pos >= 0;
        Raw<T> x[kRows], y[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int h = at.head0 + r * kSub + sub;
            x[r].zero();
            y[r].zero();
            if (h < heads && c.in) {
                const char* row = in.p + t * in.ts + h * in.hs;
                x[r].load(row + c.e0 * sizeof(T));
                if (!kInter && c.any && turned) load_partner<T, kInter>(y[r], row, c, p.rot);
            }
        }
        float co[8], si[8];
        load_angles<kInter>(co, si, c, p, pos, turned);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            co[k] *= wj[k];
            si[k] *= wo[k];
        }
        __syncwarp();  // rows may be overwritten in place: all of a row is read by now
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int h = at.head0 + r * kSub + sub;
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s = fmaf(x[r].get(k), x[r].get(k), s);
            s = row_sum<kLanes>(s);
            const float rn = rsqrtf(fmaf(s, inv_dim, p.eps));
            if (h < heads && c.in) {
                float o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float other = 0.f;
                    if (kInter) {
                        if (turned && c.e0 + k < p.rot) other = x[r].get(k ^ 1);
                    } else {
                        other = y[r].get(k);
                    }
                    o[k] = rn * fmaf(other, si[k], x[r].get(k) * co[k]);
                }
                Raw<T>::store(out.p + t * out.ts + h * out.hs + c.e0 * sizeof(T), o);
            }
        }
    }
}

template <typename T, bool kInter, int kLanes, int kRows>
__global__ void __launch_bounds__(kHnThreads) headnorm_bwd_kernel(const HnParams p) {
    grid_dep_sync();
    constexpr int kSub = 32 / kLanes;
    __shared__ float sum[kHnWarps][kLanes * 8];
    __shared__ bool of_keys[kHnWarps];
    const Place at = place<kSub * kRows>(p);
    const int lane = threadIdx.x & (kLanes - 1), sub = (threadIdx.x & 31) / kLanes;
    const int warp = threadIdx.x >> 5;
    const Cols c = columns<kInter>(lane, p.dim, p.rot);
    float dw[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[k] = 0.f;
    if (at.active) {
        const Rows in = at.keys ? p.k : p.q, gy = at.keys ? p.yk : p.yq, out = at.keys ? p.dk : p.dq;
        const int heads = at.keys ? p.hk : p.hq;
        const float* w = at.keys ? p.kw : p.qw;
        float wj[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) wj[k] = w && c.in ? __ldg(w + c.e0 + k) : 1.f;
        const float inv_dim = 1.f / (float)p.dim;
        for (int64_t t = at.token; t < p.tokens; t += at.step) {
            const int64_t pos = p.positions ? (int64_t)__ldg(p.positions + t) : t;
            const bool turned = pos >= 0;
            Raw<T> x[kRows], d[kRows], y[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int h = at.head0 + r * kSub + sub;
                x[r].zero();
                d[r].zero();
                y[r].zero();
                if (h < heads && c.in) {
                    x[r].load(in.p + t * in.ts + h * in.hs + c.e0 * sizeof(T));
                    const char* row = gy.p + t * gy.ts + h * gy.hs;
                    d[r].load(row + c.e0 * sizeof(T));
                    if (!kInter && c.any && turned) load_partner<T, kInter>(y[r], row, c, p.rot);
                }
            }
            float co[8], si[8];
            load_angles<kInter>(co, si, c, p, pos, turned);
            __syncwarp();  // the gradient may be written over dy or x
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int h = at.head0 + r * kSub + sub;
                float g[8], s = 0.f, dot = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float other = 0.f;
                    if (kInter) {
                        if (turned && c.e0 + k < p.rot) other = d[r].get(k ^ 1);
                    } else {
                        other = y[r].get(k);
                    }
                    g[k] = fmaf(-other, si[k], d[r].get(k) * co[k]);
                    const float xv = x[r].get(k);
                    s = fmaf(xv, xv, s);
                    dot = fmaf(wj[k] * g[k], xv, dot);
                }
                s = row_sum<kLanes>(s);
                dot = row_sum<kLanes>(dot);
                const float rn = rsqrtf(fmaf(s, inv_dim, p.eps));
                const float m = dot * inv_dim * rn * rn;
                if (h < heads && c.in) {
                    float o[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float xv = x[r].get(k);
                        o[k] = rn * fmaf(-xv, m, wj[k] * g[k]);
                        dw[k] = fmaf(g[k], xv * rn, dw[k]);
                    }
                    Raw<T>::store(out.p + t * out.ts + h * out.hs + c.e0 * sizeof(T), o);
                }
            }
        }
    }
    // the warp's rows, then the block's warps of the same side, in order
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], o);
        if (sub == 0) sum[warp][lane * 8 + k] = dw[k];
    }
    if ((threadIdx.x & 31) == 0) of_keys[warp] = at.keys;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.dim; i += kHnThreads) {
        const bool keys = i >= p.dim;
        const int e = keys ? i - p.dim : i;
        float s = 0.f;
        for (int v = 0; v < kHnWarps; ++v)
            if (of_keys[v] == keys) s += sum[v][e];
        p.part[(int64_t)blockIdx.x * 2 * p.dim + i] = s;
    }
}

// dw[side][e] = the blocks' sums in block order: 8 threads take every 8th block of a
// column, their sums are added in order
__global__ void __launch_bounds__(kHnThreads)
    headnorm_finish_kernel(const float* __restrict__ part, int blocks, int dim, float* dqw,
                           float* dkw) {
    grid_dep_sync();
    __shared__ float s[kHnThreads / kFinishCols][kFinishCols];
    const int col = threadIdx.x % kFinishCols, row = threadIdx.x / kFinishCols;
    const int i = blockIdx.x * kFinishCols + col;
    float a = 0.f;
    if (i < 2 * dim)
#pragma unroll 8
        for (int b = row; b < blocks; b += kHnThreads / kFinishCols)
            a += __ldg(part + (int64_t)b * 2 * dim + i);
    s[row][col] = a;
    __syncthreads();
    if (row == 0 && i < 2 * dim) {
        for (int r = 1; r < kHnThreads / kFinishCols; ++r) a += s[r][col];
        float* out = i < dim ? dqw : dkw;
        if (out) out[i < dim ? i : i - dim] = a;
    }
}

Rows rows_of(const gs_heads& h, int size) {
    return {static_cast<char*>(h.data), h.token_stride * size, h.head_stride * size};
}

int lanes_of(int dim) {
    int lanes = 1;
    while (lanes * 8 < dim) lanes *= 2;
    return lanes;
}

// Rows in flight per lane: 4 of bfloat16; 2 of fp32, whose rows take twice the registers.
constexpr int kRows16 = 4, kRows32 = 2;

template <typename T, bool kInter, int kLanes>
cudaError_t launch_lanes(HnParams p, bool bwd, int* blocks_out, cudaStream_t st) {
    constexpr int kRows = sizeof(T) == 2 ? kRows16 : kRows32;
    constexpr int kHeads = 32 / kLanes * kRows;
    p.chunks_q = (p.hq + kHeads - 1) / kHeads;
    p.chunks_k = (p.hk + kHeads - 1) / kHeads;
    const int64_t chunks = p.chunks_q + p.chunks_k;
    const int64_t want = (p.tokens * chunks + kHnWarps - 1) / kHnWarps;
    const int64_t least = (chunks + kHnWarps - 1) / kHnWarps;
    const int blocks = (int)std::max(least, std::min<int64_t>(want, kHnMaxBlocks));
    *blocks_out = blocks;
    if (bwd)
        return launch(headnorm_bwd_kernel<T, kInter, kLanes, kRows>, dim3(blocks),
                      dim3(kHnThreads), 0, st, p);
    return launch(headnorm_kernel<T, kInter, kLanes, kRows>, dim3(blocks), dim3(kHnThreads), 0, st,
                  p);
}

template <typename T, bool kInter>
cudaError_t launch_typed(const HnParams& p, bool bwd, int* blocks, cudaStream_t st) {
    switch (lanes_of(p.dim)) {
        case 1: return launch_lanes<T, kInter, 1>(p, bwd, blocks, st);
        case 2: return launch_lanes<T, kInter, 2>(p, bwd, blocks, st);
        case 4: return launch_lanes<T, kInter, 4>(p, bwd, blocks, st);
        case 8: return launch_lanes<T, kInter, 8>(p, bwd, blocks, st);
        case 16: return launch_lanes<T, kInter, 16>(p, bwd, blocks, st);
        default: return launch_lanes<T, kInter, 32>(p, bwd, blocks, st);
    }
}

cudaError_t launch_any(const HeadNormArgs& a, const HnParams& p, bool bwd, int* blocks,
                       cudaStream_t st) {
    if (a.bf16)
        return a.interleaved ? launch_typed<__nv_bfloat16, true>(p, bwd, blocks, st)
                             : launch_typed<__nv_bfloat16, false>(p, bwd, blocks, st);
    return a.interleaved ? launch_typed<float, true>(p, bwd, blocks, st)
                         : launch_typed<float, false>(p, bwd, blocks, st);
}

HnParams params_of(const HeadNormArgs& a, const gs_heads& q, const gs_heads& k,
                   const gs_heads& yq, const gs_heads& yk) {
    const int size = a.bf16 ? 2 : 4;
    HnParams p{};
    p.tokens = a.tokens;
    p.table_rows = a.table_rows;
    p.hq = a.hq;
    p.hk = a.hk;
    p.dim = a.dim;
    p.rot = a.rot;
    p.eps = a.eps;
    p.qw = a.qw;
    p.kw = a.kw;
    p.cos_sin = a.cos_sin;
    p.positions = a.positions;
    p.q = rows_of(q, size);
    p.k = rows_of(k, size);
    p.yq = rows_of(yq, size);
    p.yk = rows_of(yk, size);
    return p;
}

}  // namespace

size_t headnorm_workspace_bytes(int64_t tokens, int dim) {
    (void)tokens;
    return (size_t)kHnMaxBlocks * 2 * dim * sizeof(float);
}

cudaError_t launch_headnorm(const HeadNormArgs& a, const gs_heads& q, const gs_heads& k,
                            const gs_heads& q_out, const gs_heads& k_out, cudaStream_t st) {
    int blocks = 0;
    return launch_any(a, params_of(a, q, k, q_out, k_out), false, &blocks, st);
}

cudaError_t launch_headnorm_bwd(const HeadNormArgs& a, const gs_heads& q, const gs_heads& k,
                                const gs_heads& dq_out, const gs_heads& dk_out,
                                const gs_heads& dq, const gs_heads& dk, float* dqw, float* dkw,
                                void* ws, cudaStream_t st) {
    HnParams p = params_of(a, q, k, dq_out, dk_out);
    const int size = a.bf16 ? 2 : 4;
    p.dq = rows_of(dq, size);
    p.dk = rows_of(dk, size);
    p.part = static_cast<float*>(ws);
    int blocks = 0;
    const cudaError_t e = launch_any(a, p, true, &blocks, st);
    if (e != cudaSuccess || (!dqw && !dkw)) return e;
    return launch(headnorm_finish_kernel, dim3((2 * a.dim + kFinishCols - 1) / kFinishCols),
                  dim3(kHnThreads), 0, st, static_cast<const float*>(p.part), blocks, a.dim, dqw,
                  dkw);
}

}  // namespace gs
