// gs_clip.cu -- the norm over many arrays of gradients and their scaling to at most a given norm.
//
//   norm = (sum over all arrays of g^2)^(1/2),  out = g min(1, max_norm / norm)
//
// Two kernels.  The first sums squares, the second joins the blocks' sums (each of its blocks for
// itself: at most kBlocks numbers a table, from L2) and scales.  The arrays travel as a table in the
// kernel's parameters, so nothing is copied to the device beforehand and a captured graph keeps its
// own.  A block takes chunks of kChunkBytes in turn and finds a chunk's array by bisection.
//
// Memory bounds it: the arrays are read, then read and written.  The second kernel walks the
// chunks backwards, so that it meets first what the first one left in L2.
//
// Sums.  A thread's squares of one chunk (at most 64) go into fp32, the chunks' sums into fp64:
// 1.7e12 fp32 elements arrive a second, fp64 units take a third of that.  Squares leave the range
// of fp32 long before their root does, so a sum outside [2^-100, 2^126] is formed again in fp64
// from the values still in registers (zeros, which whole arrays may hold, are told apart first).
// Blocks and chunks go in a fixed order: the same inputs give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gs_device.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {
namespace {

constexpr int kClipThreads = 256;
constexpr int kVecs = 4;  // 16-byte words a thread takes of a chunk
constexpr int kChunkBytes = kClipThreads * kVecs * 16;
constexpr int kBlocks = 152 * 6;  // resident at once
constexpr int kFewArrays = 96, kManyArrays = 1024;  // of a table: 3 KB and 29 KB of parameters
constexpr int kMaxTables = 64;

template <int kArrays>
struct Table {
    int64_t elements[kArrays];  // bit 62: bfloat16
    const void* in[kArrays];
    void* out[kArrays];
    int32_t chunk0[kArrays + 1];  // first chunk of each
    int count;
};
constexpr int64_t kBf16Bit = int64_t(1) << 62;

struct Chunk {
    const char* in;
    char* out;
    int elements;  // of the chunk
    bool bf16;
};

template <int kArrays>
__device__ __forceinline__ Chunk chunk_of(const Table<kArrays>& t, int id) {
    int lo = 0, hi = t.count;  // the last array that starts at the chunk or before (empty ones before it)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.chunk0[mid] <= id)
            lo = mid;
        else
            hi = mid;
    }
    const int64_t n = t.elements[lo] & ~kBf16Bit;
    const bool bf16 = t.elements[lo] & kBf16Bit;
    const int per = kChunkBytes / (bf16 ? 2 : 4);
    const int64_t first = (int64_t)(id - t.chunk0[lo]) * per;
    return {static_cast<const char*>(t.in[lo]) + first * (bf16 ? 2 : 4),
            static_cast<char*>(t.out[lo]) + first * (bf16 ? 2 : 4), (int)min64(n - first, per), bf16};
}

__device__ __forceinline__ bool words16(const void* p) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// sum of the squares of a thread's values
template <int kN>
__device__ __forceinline__ double squares(const float (&v)[kN]) {
    float2 s = make_float2(0.f, 0.f), u = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kN; k += 4) {
        const float2 a = make_float2(v[k], v[k + 1]), b = make_float2(v[k + 2], v[k + 3]);
        s = __ffma2_rn(a, a, s);
        u = __ffma2_rn(b, b, u);
    }
    const float sum = (s.x + s.y) + (u.x + u.y);
    if (sum >= 0x1p-100f && sum <= 0x1p126f) return (double)sum;
    float top = 0.f;
    bool other = false;  // NaN
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        top = fmaxf(top, fabsf(v[k]));
        other |= v[k] != v[k];
    }
    if (top == 0.f && !other) return 0.0;
    double d = 0.0;
#pragma unroll
    for (int k = 0; k < kN; ++k) d = fma((double)v[k], (double)v[k], d);
    return d;
}

// the block's sum, to thread 0: lanes, then warps in order
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double of_warp[kClipThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kClipThreads / 32; ++w) v += of_warp[w];
    return v;
}

template <int kArrays>
__global__ void __launch_bounds__(kClipThreads, 6)
    square_sum_kernel(const __grid_constant__ Table<kArrays> t, double* part) {
    grid_dep_sync();
    const int chunks = t.chunk0[t.count];
    double sum = 0.0;
    for (int id = blockIdx.x; id < chunks; id += gridDim.x) {
        const Chunk c = chunk_of(t, id);
        const bool whole = c.elements * (c.bf16 ? 2 : 4) == kChunkBytes && words16(c.in);
        if (whole) {
            uint4 w[kVecs];
#pragma unroll
            for (int k = 0; k < kVecs; ++k)
                w[k] = __ldg(reinterpret_cast<const uint4*>(c.in) + k * kClipThreads + threadIdx.x);
            if (c.bf16) {
                float v[8 * kVecs];
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[8 * k + 2 * e] = lo16(u[e]);
                        v[8 * k + 2 * e + 1] = hi16(u[e]);
                    }
                }
                sum += squares(v);
            } else {
                float v[4 * kVecs];
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    v[4 * k] = __uint_as_float(w[k].x);
                    v[4 * k + 1] = __uint_as_float(w[k].y);
                    v[4 * k + 2] = __uint_as_float(w[k].z);
                    v[4 * k + 3] = __uint_as_float(w[k].w);
                }
                sum += squares(v);
            }
            continue;
        }
        // an array's end, or one that does not start at a word: element by element
        for (int e0 = 0; e0 < c.elements; e0 += 4 * kClipThreads) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int e = e0 + k * kClipThreads + threadIdx.x;
                v[k] = 0.f;
                if (e < c.elements)
                    v[k] = c.bf16 ? lo16(reinterpret_cast<const uint16_t*>(c.in)[e])
                                  : reinterpret_cast<const float*>(c.in)[e];
            }
            sum += squares(v);
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// A value times the factor.  A factor below fp32's normal range has lost bits: fp64 then (kTiny; not
// chosen value by value, which would cost the fp64 units' time always).
template <bool kTiny>
__device__ __forceinline__ float scaled(float v, double d) {
    return kTiny ? (float)((double)v * d) : v * (float)d;
}

__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kTiny>
__device__ __forceinline__ void scale_chunk(const Chunk& c, double d) {
    const bool whole = c.elements * (c.bf16 ? 2 : 4) == kChunkBytes && words16(c.in) && words16(c.out);
    if (whole) {
        const uint4* in = reinterpret_cast<const uint4*>(c.in) + threadIdx.x;
        uint4* out = reinterpret_cast<uint4*>(c.out) + threadIdx.x;
        uint4 w[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            w[k] = d != 0.0 ? __ldcs(in + k * kClipThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                u[e] = c.bf16 ? pair_bf16(scaled<kTiny>(lo16(u[e]), d), scaled<kTiny>(hi16(u[e]), d))
                              : __float_as_uint(scaled<kTiny>(__uint_as_float(u[e]), d));
            __stcs(out + k * kClipThreads, make_uint4(u[0], u[1], u[2], u[3]));
        }
        return;
    }
    for (int e = threadIdx.x; e < c.elements; e += kClipThreads) {
        if (c.bf16) {
            const float v = d != 0.0 ? lo16(reinterpret_cast<const uint16_t*>(c.in)[e]) : 0.f;
            reinterpret_cast<__nv_bfloat16*>(c.out)[e] = __float2bfloat16_rn(scaled<kTiny>(v, d));
        } else {
            const float v = d != 0.0 ? reinterpret_cast<const float*>(c.in)[e] : 0.f;
            reinterpret_cast<float*>(c.out)[e] = scaled<kTiny>(v, d);
        }
    }
}

// A table without arrays gives the norm alone.
template <int kArrays>
__global__ void __launch_bounds__(kClipThreads, 6)
    clip_kernel(const __grid_constant__ Table<kArrays> t, const double* __restrict__ part, int parts,
                double max_norm, float* norm_out) {
    grid_dep_sync();
    __shared__ double total;
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kClipThreads) sum += __ldg(part + i);
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        if (norm_out && blockIdx.x == 0) *norm_out = (float)norm;
        // 0 where the norm is not finite: nothing is read then
        total = !(norm < INFINITY) ? 0.0 : norm > max_norm ? max_norm / norm : 1.0;
    }
    __syncthreads();
    const double d = total;
    const int chunks = t.chunk0[t.count];
    for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
        const Chunk c = chunk_of(t, chunks - 1 - i);
        if (c.in == c.out && d == 1.0) continue;
        if (d == 0.0 || d >= 0x1p-126)
            scale_chunk<false>(c, d);
        else
            scale_chunk<true>(c, d);
    }
}

// The arrays from `first` on as a table, as many as it holds; returns the one behind them.
// (Their chunks stay in 32 bits: at most 2^42 elements in all.)
template <int kArrays>
int fill(Table<kArrays>* t, int first, int count, const gs_array* in, const gs_array* out) {
    int n = 0, i = first;
    int32_t chunks = 0;
    for (; i < count && n < kArrays; ++i) {
        if (in[i].elements == 0) continue;
        const bool bf16 = in[i].type == GS_TYPE_BF16;
        t->elements[n] = in[i].elements | (bf16 ? kBf16Bit : 0);
        t->in[n] = in[i].data;
        t->out[n] = out[i].data;
        t->chunk0[n++] = chunks;
        const int64_t per = kChunkBytes / (bf16 ? 2 : 4);
        chunks += (int32_t)((in[i].elements + per - 1) / per);
    }
    t->count = n;
    t->chunk0[n] = chunks;
    return i;
}

template <int kArrays>
unsigned blocks_of(const Table<kArrays>& t) {
    return (unsigned)std::min(std::max(t.chunk0[t.count], 1), kBlocks);
}

template <int kArrays>
cudaError_t launch_tables(int count, const gs_array* in, const gs_array* out, double max_norm,
                          float* norm, double* part, cudaStream_t st) {
    Table<kArrays> t;
    int starts[kMaxTables], tables = 0, parts = 0, next = 0;
    do {
        starts[tables++] = next;
        next = fill(&t, next, count, in, out);
        const unsigned blocks = blocks_of(t);
        const cudaError_t e = launch(square_sum_kernel<kArrays>, dim3(blocks), dim3(kClipThreads), 0,
                                     st, t, part + parts);
        if (e != cudaSuccess) return e;
        parts += (int)blocks;
    } while (next < count);
    // from the last table on, which is still filled: what was read last is still in L2
    for (int i = tables - 1; i >= 0; --i) {
        if (i < tables - 1) fill(&t, starts[i], count, in, out);
        const cudaError_t e =
            launch(clip_kernel<kArrays>, dim3(blocks_of(t)), dim3(kClipThreads), 0, st, t,
                   (const double*)part, parts, max_norm, i == 0 ? norm : (float*)nullptr);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t clip_workspace_bytes(int count) {
    const int tables = std::max(1, (count + kManyArrays - 1) / kManyArrays);
    return (size_t)tables * kBlocks * sizeof(double);
}

// A table of few arrays keeps the launches' parameters short.
cudaError_t launch_clip(int count, const gs_array* in, const gs_array* out, double max_norm,
                        float* norm, void* ws, cudaStream_t st) {
    double* part = static_cast<double*>(ws);
    return count <= kFewArrays
               ? launch_tables<kFewArrays>(count, in, out, max_norm, norm, part, st)
               : launch_tables<kManyArrays>(count, in, out, max_norm, norm, part, st);
}

}  // namespace gs
