// gs_dropout.cu -- out = residual + dropout(x), with the mask from a counter-based
// generator and never stored: the backward makes it again.
//
// Element e belongs to group i = e / 8; Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with key = the seed
// and counter = (i, offset), both 64 bits, gives the group 128 bits, 16 for each
// element in order.  The element is dropped iff its 16 bits are below
// `dropped` = round(65536 p), and the others are scaled by 65536 / (65536 -
// dropped), the reciprocal of the probability actually held, so that the mean is
// kept exactly.  16 bits instead of 32 halve the generator's work: ten rounds of
// two wide products for eight elements, about 12 integer operations an element,
// which stay under the time of the element's bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gs_device.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {
namespace {

constexpr int kDropThreads = 256;

struct Words {
    uint32_t w[4];
};

__device__ __forceinline__ Words philox4x32_10(uint64_t counter_lo, uint64_t counter_hi,
                                               uint64_t key) {
    uint32_t c0 = (uint32_t)counter_lo, c1 = (uint32_t)(counter_lo >> 32);
    uint32_t c2 = (uint32_t)counter_hi, c3 = (uint32_t)(counter_hi >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return {{c0, c1, c2, c3}};
}

// eight values at element 8 i, `full` of them in range
template <typename T>
struct Eight;

template <>
struct Eight<float> {
    __device__ static void load(float (&v)[8], const float* p) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
        const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ static void store(float* p, const float (&v)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ static float get(const float* p) { return *p; }
    __device__ static void put(float* p, float v) { *p = v; }
};

template <>
struct Eight<__nv_bfloat16> {
    __device__ static void load(float (&v)[8], const __nv_bfloat16* p) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    __device__ static void store(__nv_bfloat16* p, const float (&v)[8]) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
    }
    __device__ static float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    __device__ static void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

// A thread makes the mask of one group; out may be x or residual itself (each
// element is read before it is written, by the same thread).
template <typename T, bool kResidual>
__global__ void __launch_bounds__(kDropThreads)
    dropout_add_kernel(int64_t n, const T* x, const T* residual, T* out,
                       const int64_t* __restrict__ rng, uint32_t dropped, float scale) {
    grid_dep_sync();
    const int64_t i = (int64_t)blockIdx.x * kDropThreads + threadIdx.x;
    const int64_t e = i * 8;
    if (e >= n) return;
    const Words w = philox4x32_10((uint64_t)i, (uint64_t)__ldg(rng + 1), (uint64_t)__ldg(rng));
    bool keep[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t bits = (k & 1) ? w.w[k >> 1] >> 16 : w.w[k >> 1] & 0xffffu;
        keep[k] = bits >= dropped;
    }
    if (e + 8 <= n) {
        float v[8], y[8];
        Eight<T>::load(v, x + e);
        if (kResidual) Eight<T>::load(y, residual + e);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // a dropped value counts as 0 whatever it was, infinities and NaN included
            const float r = kResidual ? y[k] : 0.f;
            v[k] = keep[k] ? fmaf(v[k], scale, r) : r;
        }
        Eight<T>::store(out + e, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (e + k >= n) break;
            const float r = kResidual ? Eight<T>::get(residual + e + k) : 0.f;
            Eight<T>::put(out + e + k,
                          keep[k] ? fmaf(Eight<T>::get(x + e + k), scale, r) : r);
        }
    }
}

template <typename T>
cudaError_t launch_typed(int64_t n, const void* x, const void* residual, void* out,
                         const int64_t* rng, uint32_t dropped, cudaStream_t st) {
    const float scale = (float)(65536.0 / (65536.0 - dropped));
    const dim3 grid((unsigned)((n + 8 * kDropThreads - 1) / (8 * kDropThreads)));
    const T *xt = static_cast<const T*>(x), *rt = static_cast<const T*>(residual);
    if (residual)
        return launch(dropout_add_kernel<T, true>, grid, dim3(kDropThreads), 0, st, n, xt, rt,
                      static_cast<T*>(out), rng, dropped, scale);
    return launch(dropout_add_kernel<T, false>, grid, dim3(kDropThreads), 0, st, n, xt, rt,
                  static_cast<T*>(out), rng, dropped, scale);
}

}  // namespace

cudaError_t launch_dropout_add(int64_t n, bool bf16, const void* x, const void* residual,
                               void* out, const int64_t* rng, uint32_t dropped, cudaStream_t st) {
    return bf16 ? launch_typed<__nv_bfloat16>(n, x, residual, out, rng, dropped, st)
                : launch_typed<float>(n, x, residual, out, rng, dropped, st);
}

}  // namespace gs
