// gs_clip.cu -- the norm over many arrays of gradients and their scaling to at most a given norm.
//
//   norm = (sum over all arrays of g^2)^(1/2),  out = g min(1, max_norm / norm)
//
// Two kernels.  The first sums squares, the second joins the blocks' sums (each of its blocks for
// itself: at most kBlocks numbers a table, from L2, while its first chunk is on its way) and scales.
// The arrays travel as a table in the kernel's parameters, so nothing is copied to the device
// beforehand and a captured graph keeps its own.  A block takes neighbouring chunks of kChunkBytes;
// the table tells it the array of the first one (a search through the arrays would be one miss of
// the constant cache after the other).
//
// Memory bounds it: the arrays are read, then read and written.  The second kernel walks a block's
// chunks backwards, so that it meets first what the first one left in L2.  88.5M fp32 values: 169 us,
// 6.3 TB/s of three times their bytes; 139M bfloat16 ones 143 us; 2.4M fp32 ones (L2 holds them) 11.1 us,
// the latency of two kernels and of the arrays' ends, which go element by element.
//
// Sums.  A thread's squares of one chunk (at most 64) go into fp32, the chunks' sums into pairs of
// fp32 (a sum and what its roundings left), the blocks' into fp64, whose units take a third of the
// 1.7e12 fp32 elements that arrive a second.  Squares leave the range of fp32 long before their root
// does, so a chunk's sum outside [2^-90, 2^80] is formed again in fp64 from the values still in
// registers (zeros, which whole arrays may hold, are told apart first).  Blocks and chunks go in a
// fixed order: the same inputs give the same bits.
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
// Four blocks an SM and chunks of 32 KB (six and 16 KB: 12.6 us instead of 11.0 on 2.4M fp32 values,
// 181 instead of 175 on 88.5M, all read alike).
constexpr int kVecs = 8;  // 16-byte words a thread takes of a chunk
constexpr int kChunkBytes = kClipThreads * kVecs * 16;
constexpr int kBlocks = 152 * 4;  // resident at once
// What is to stay in L2 from the first kernel to the second.  (Half of L2; 88.5M fp32 values: 175 us
// where all is read alike, 171 with 40 MB, 169 with 64 and 96.)
constexpr int64_t kKeptBytes = 64 << 20;
constexpr int kFewArrays = 96, kManyArrays = 1024;  // of a table: 5 KB and 31 KB of parameters
constexpr int kMaxTables = 64;

template <int kArrays>
struct Table {
    int64_t elements[kArrays];  // bit 62: bfloat16
    const void* in[kArrays];
    void* out[kArrays];
    int32_t chunk0[kArrays + 1];  // first chunk of each
    int count;
    uint16_t first[kBlocks + 1];  // array of each block's first chunk; the last array
};
constexpr int64_t kBf16Bit = int64_t(1) << 62;

// first chunk of block b of `blocks`
__host__ __device__ __forceinline__ int first_chunk(int chunks, int blocks, int b) {
    return (int)((int64_t)chunks * b / blocks);
}

struct Chunk {
    const char* in;
    char* out;
    int elements;  // of the chunk
    bool bf16;
};

// chunk `id`, of array i
template <int kArrays>
__device__ __forceinline__ Chunk chunk_of(const Table<kArrays>& t, int i, int id) {
    const int64_t n = t.elements[i] & ~kBf16Bit;
    const bool bf16 = t.elements[i] & kBf16Bit;
    const int per = kChunkBytes / (bf16 ? 2 : 4);
    const int64_t first = (int64_t)(id - t.chunk0[i]) * per;
    return {static_cast<const char*>(t.in[i]) + first * (bf16 ? 2 : 4),
            static_cast<char*>(t.out[i]) + first * (bf16 ? 2 : 4), (int)min64(n - first, per), bf16};
}

__device__ __forceinline__ bool words16(const void* p) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A sum as two floats, and what lies outside fp32's range apart.
struct Sum {
    float high = 0.f, low = 0.f;
    double odd = 0.0;
    __device__ __forceinline__ void add(float v, float v_low) {  // Knuth's sum and its rounding
        const float s = high + v, b = s - high;
        low += ((high - (s - b)) + (v - b)) + v_low;
        high = s;
    }
    // the squares of a thread's values
    template <int kN>
    __device__ __forceinline__ void squares(const float (&v)[kN]) {
        float2 s = make_float2(0.f, 0.f), u = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kN; k += 4) {
            const float2 a = make_float2(v[k], v[k + 1]), b = make_float2(v[k + 2], v[k + 3]);
            s = __ffma2_rn(a, a, s);
            u = __ffma2_rn(b, b, u);
        }
        const float sum = (s.x + s.y) + (u.x + u.y);
        if (sum >= 0x1p-90f && sum <= 0x1p80f) {
            add(sum, 0.f);
            return;
        }
        float top = 0.f;
        bool other = false;  // NaN
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            top = fmaxf(top, fabsf(v[k]));
            other |= v[k] != v[k];
        }
        if (top == 0.f && !other) return;
#pragma unroll
        for (int k = 0; k < kN; ++k) odd = fma((double)v[k], (double)v[k], odd);
    }
};

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

__device__ __forceinline__ double block_sum(Sum s) {
    __shared__ float2 of_warp[kClipThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float high = __shfl_xor_sync(0xffffffffu, s.high, o);
        s.add(high, __shfl_xor_sync(0xffffffffu, s.low, o));
    }
    if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = make_float2(s.high, s.low);
    const bool odd = __syncthreads_or(s.odd != 0.0);
    double v = 0.0;
    if (threadIdx.x == 0) {
        Sum all;
        for (int w = 0; w < kClipThreads / 32; ++w) all.add(of_warp[w].x, of_warp[w].y);
        v = (double)all.high + (double)all.low;
    }
    return odd ? v + block_sum(s.odd) : v;
}

template <int kArrays>
__global__ void __launch_bounds__(kClipThreads, 4)
    square_sum_kernel(const __grid_constant__ Table<kArrays> t, double* part) {
    grid_dep_sync();
    const int chunks = t.chunk0[t.count];
    const int end = first_chunk(chunks, gridDim.x, blockIdx.x + 1);
    // the last chunks, which the second kernel takes first; the others are the first to leave L2
    const int kept =
        end - max(1, (int)(kKeptBytes / ((int64_t)gridDim.x * kChunkBytes)));
    int array = t.first[blockIdx.x];
    Sum sum;
    for (int id = first_chunk(chunks, gridDim.x, blockIdx.x); id < end; ++id) {
        while (t.chunk0[array + 1] <= id) ++array;
        const Chunk c = chunk_of(t, array, id);
        const bool whole = c.elements * (c.bf16 ? 2 : 4) == kChunkBytes && words16(c.in);
        if (whole) {
            uint4 w[kVecs];
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const uint4* from =
                    reinterpret_cast<const uint4*>(c.in) + k * kClipThreads + threadIdx.x;
                w[k] = id >= kept ? __ldg(from) : __ldcs(from);
            }
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
                sum.squares(v);
            } else {
                float v[4 * kVecs];
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    v[4 * k] = __uint_as_float(w[k].x);
                    v[4 * k + 1] = __uint_as_float(w[k].y);
                    v[4 * k + 2] = __uint_as_float(w[k].z);
                    v[4 * k + 3] = __uint_as_float(w[k].w);
                }
                sum.squares(v);
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
            sum.squares(v);
        }
    }
    const double total = block_sum(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = total;
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

__device__ __forceinline__ bool whole_chunk(const Chunk& c) {
    return c.elements * (c.bf16 ? 2 : 4) == kChunkBytes && words16(c.in) && words16(c.out);
}

// a thread's words of a whole chunk
struct ChunkWords {
    uint4 w[kVecs];
    __device__ __forceinline__ void load(const Chunk& c) {
        const uint4* in = reinterpret_cast<const uint4*>(c.in) + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) w[k] = __ldcs(in + k * kClipThreads);
    }
};

template <bool kTiny>
__device__ __forceinline__ void scale_chunk(const Chunk& c, const ChunkWords& x, bool whole, double d) {
    if (whole) {
        uint4* out = reinterpret_cast<uint4*>(c.out) + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            uint32_t u[4] = {x.w[k].x, x.w[k].y, x.w[k].z, x.w[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (c.bf16)
                    u[e] = pair_bf16(scaled<kTiny>(lo16(u[e]), d), scaled<kTiny>(hi16(u[e]), d));
                else
                    u[e] = __float_as_uint(scaled<kTiny>(__uint_as_float(u[e]), d));
                if (d == 0.0) u[e] = 0;  // whatever the gradient is
            }
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
__global__ void __launch_bounds__(kClipThreads, 4)
    clip_kernel(const __grid_constant__ Table<kArrays> t, const double* __restrict__ part, int parts,
                double max_norm, float* norm_out) {
    grid_dep_sync();
    __shared__ double total;
    const int chunks = t.chunk0[t.count];
    const int begin = first_chunk(chunks, gridDim.x, blockIdx.x);
    int id = first_chunk(chunks, gridDim.x, blockIdx.x + 1) - 1, array = t.first[blockIdx.x + 1];
    Chunk c{};
    ChunkWords x;
    bool whole = false;
    const auto load = [&](bool same) {  // same: chunks that stay in their place are not read
        if (id < begin) return;
        while (t.chunk0[array] > id) --array;
        c = chunk_of(t, array, id);
        whole = whole_chunk(c);
        if (whole && !(same && c.in == c.out)) x.load(c);
    };
    load(false);
    // (the first chunk is on its way before the factor is known)
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kClipThreads) sum += __ldg(part + i);
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        // in fp32, whose root and quotient take a tenth of fp64's time, where both are in its range
        if (sum >= 0x1p-100 && sum <= 0x1p126) {
            const float norm = __fsqrt_rn((float)sum);
            if (norm_out && blockIdx.x == 0) *norm_out = norm;
            total = !(norm > max_norm)  ? 1.0
                    : max_norm >= 0x1p-60 ? (double)__fdiv_rn((float)max_norm, norm)
                                          : max_norm / norm;
        } else {
            const double norm = sqrt(sum);
            if (norm_out && blockIdx.x == 0) *norm_out = (float)norm;
            // 0 where the norm is not finite, unless all is wanted as it is
            total = max_norm == INFINITY  ? 1.0
                    : !(norm < INFINITY)  ? 0.0
                    : norm > max_norm     ? max_norm / norm
                                          : 1.0;
        }
    }
    __syncthreads();
    const double d = total;
    for (; id >= begin; --id, load(d == 1.0)) {
        if (c.in == c.out && d == 1.0) continue;
        if (d == 0.0 || d >= 0x1p-126)
            scale_chunk<false>(c, x, whole, d);
        else
            scale_chunk<true>(c, x, whole, d);
    }
}

template <int kArrays>
unsigned blocks_of(const Table<kArrays>& t) {
    return (unsigned)std::min(std::max(t.chunk0[t.count], 1), kBlocks);
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
    const int blocks = (int)blocks_of(*t);
    for (int b = 0, a = 0; b < blocks; ++b) {
        while (a + 1 < n && t->chunk0[a + 1] <= first_chunk(chunks, blocks, b)) ++a;
        t->first[b] = (uint16_t)a;
    }
    t->first[blocks] = (uint16_t)(n > 0 ? n - 1 : 0);
    return i;
}

template <int kArrays>
cudaError_t launch_tables(int count, const gs_array* in, const gs_array* out, double max_norm,
                          float* norm, double* part, cudaStream_t st) {
    bool alone = max_norm == INFINITY;  // the norm alone is wanted
    for (int i = 0; i < count && alone; ++i) alone = in[i].data == out[i].data;
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
    if (alone) {
        fill(&t, 0, 0, in, out);
        return launch(clip_kernel<kArrays>, dim3(1), dim3(kClipThreads), 0, st, t, (const double*)part,
                      parts, max_norm, norm);
    }
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
