// gs_residual_norm.cu -- what stands between two blocks of a network in one pass: the norm of a
// block's output, its gate and scale, the residual, and the norm before the next block; and the
// gradient of it all.
//
//   u = post(y),  r = alpha x + beta gate u,  h = pre(r)
//
// with norm(v) = w (v - m) s + b, s = (mean (v - m)^2 + eps)^(-1/2), m = 0 (RMS) or the mean
// (layer).  The gradient forms the row's statistics again from x and y, which costs no more bytes
// than reading r would and is of the unrounded r, as h was.  With vn = (v - m) s the gradient by v
// of a norm whose output's is g is
//   s (k - vn mean(k vn) [- mean(k) for a layer norm]),  k = w g,
// and so, with dR = dr + that of pre:
//   dx = alpha dR,  du = beta gate dR,  dy = that of post with g = du,
//   dw = sum g vn,  db = sum g,  dgate = sum beta dR u  over a sequence's tokens.
//
// Memory bounds it: four arrays forward, six backward.  A row is one block's, eight values a thread
// held in registers from the first sum over the row to the last, so nothing is read twice; a row
// of at most 256 values is one warp's and its sums need no barrier.  Weights and gates stay in
// registers, the gate multiplied into post's weight and bias: read from L1 for every row they kept
// L1 busier than the arrays did.  A block has consecutive rows, reads the next ones while it works
// on the present one, and keeps sums of the column gradients in registers: of the weights and biases over
// all its rows, of the gate over those of a sequence.  Another kernel adds the blocks' sums up in the
// blocks' order: the same inputs give the same bits.
//
// Measured, 32,400 x 1,024 in bfloat16 with RMS norms on both sides and a gate: forward 50.4 us, 5.3
// TB/s, 0.78 of the copy rate; backward 81.6 us, 4.9 TB/s, with two or three sums over a row and 16 warps
// an SM (128 registers) on the way, and 8 us of the blocks' sums.  64 x 256: 4.2 us, the latency of a
// row.  Odd widths go value by value: 4,346 x 515 in fp32 with layer norms and biases, backward, 30.5 us.
//
// All sums and statistics are fp32, the variance from the differences to the mean.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "gs_device.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {
namespace {

constexpr int kSms = 152;
constexpr int kMostThreads = 1024;  // width <= 8,192
constexpr int kFourUpTo = 2048;  // widths up to which a thread may take four values: see pairs_of
constexpr int kFwdWarps = 32, kBwdWarps = 16;  // resident on an SM
constexpr int kMostGates = 256;     // sequences at once when the gates' gradients are added up

struct NormRows {
    char* p;
    uint32_t stride;  // bytes
    // byte `shift` of a row: one multiplication instead of a pointer and a stride in registers
    __device__ __forceinline__ char* at(uint32_t row, int shift) const {
        return p + (uint64_t)row * stride + shift;
    }
};

struct RnParams {
    int64_t tokens;
    int width, batch, pre, post;
    float alpha, beta, eps;
    const float *pw, *pb, *qw, *qb, *gate;  // pre's weight and bias, post's; gate [batch][width]
    const int32_t* cu;                      // [batch + 1] or null: one sequence of all tokens
    NormRows x, y, r, h;    // forward
    NormRows dr, dh, dx, dy;  // backward
    float* dgate;           // [batch][width] or null
    // backward: [blocks][4][width] sums of the blocks for dpw, dpb, dqw, dqb; [blocks][2][width]
    // of a block's first and last sequence where those began before it, or go on behind it
    float *part, *part_gate;
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// A thread's values of a row, in pairs (two operations an instruction).
template <int kPairs>
struct Values {
    float2 v[kPairs];
};

template <int kPairs>
__device__ __forceinline__ float dot(const Values<kPairs>& a, const Values<kPairs>& b) {
    float2 s = mul(a.v[0], b.v[0]);
#pragma unroll
    for (int k = 1; k < kPairs; ++k) s = fma2(a.v[k], b.v[k], s);
    return s.x + s.y;
}
template <int kPairs>
__device__ __forceinline__ float total(const Values<kPairs>& a) {
    float2 s = a.v[0];
#pragma unroll
    for (int k = 1; k < kPairs; ++k) s = add(s, a.v[k]);
    return s.x + s.y;
}

// A thread's columns: neighbours, or (odd widths and strides) every 32nd of its warp's.
template <bool kVec, int kPairs>
struct Columns {
    static constexpr int kPer = 2 * kPairs, kStep = kVec ? 1 : 32;
    using V = Values<kPairs>;
    int first, n;  // n: those that exist
    bool full;     // the whole warp's do

    __device__ __forceinline__ Columns(int width) {
        if (kVec) {
            first = (int)threadIdx.x * kPer;
            n = first >= width ? 0 : kPer;
            full = n > 0;
        } else {
            const int lane = threadIdx.x & 31, of_warp = ((int)threadIdx.x - lane) * kPer;
            first = of_warp + lane;
            n = first >= width ? 0 : min(kPer, (width - 1 - first) / kStep + 1);
            full = of_warp + 32 * kPer <= width;
        }
    }
    // values k of the lane, by f, where there are such columns
    template <typename F>
    __device__ __forceinline__ void each(const F& f) const {
        if (full) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) f(k);
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (k < n) f(k);
        }
    }
    // values of fp32 from w, `other` where there are none
    __device__ __forceinline__ V weights(const float* w, float other) const {
        V r;
        float* v = &r.v[0].x;
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = other;
        if (!w || n == 0) return r;
        const float* p = w + first;
        if (kVec) {
#pragma unroll
            for (int k = 0; k < kPer; k += 4) {
                const float4 a = __ldg(reinterpret_cast<const float4*>(p + k));
                v[k] = a.x, v[k + 1] = a.y, v[k + 2] = a.z, v[k + 3] = a.w;
            }
        } else {
            each([&](int k) { v[k] = __ldg(p + k * kStep); });
        }
        return r;
    }
    __device__ __forceinline__ void store(float* w, const V& r) const { store_at(w + first, r); }
    __device__ __forceinline__ void store_at(float* p, const V& r) const {  // p: at the first column
        if (n == 0) return;
        const float* v = &r.v[0].x;
        if (kVec) {
#pragma unroll
            for (int k = 0; k < kPer; k += 4)
                *reinterpret_cast<float4*>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        } else {
            each([&](int k) { p[k * kStep] = v[k]; });
        }
    }
    // zero where there is no column
    __device__ __forceinline__ void trim(V& r) const {
        if (full) return;
        float* v = &r.v[0].x;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (k >= n) v[k] = 0.f;
    }
};

// A thread's values of a row as they lie in memory, zeros where there is none.
template <typename T, bool kVec, int kPairs>
struct RawRow;

template <bool kVec, int kPairs>
struct RawRow<float, kVec, kPairs> {
    using C = Columns<kVec, kPairs>;
    using V = Values<kPairs>;
    V r;
    static constexpr int kWords = kPairs / 2;  // of 16 bytes
    __device__ __forceinline__ void clear() { r = V{}; }
    __device__ __forceinline__ void load(const char* at, const C& c) {
        float* v = &r.v[0].x;
        const float* p = reinterpret_cast<const float*>(at);
        if (kVec) {
#pragma unroll
            for (int k = 0; k < C::kPer; k += 4) {
                const float4 a = __ldcs(reinterpret_cast<const float4*>(p + k));
                v[k] = a.x, v[k + 1] = a.y, v[k + 2] = a.z, v[k + 3] = a.w;
            }
        } else {
            c.each([&](int k) { v[k] = p[k * C::kStep]; });
        }
    }
    __device__ __forceinline__ V get() const { return r; }
    __device__ static __forceinline__ void store(char* at, const V& f, const C& c) {
        c.store_at(reinterpret_cast<float*>(at), f);
    }
};

template <bool kVec, int kPairs>
struct RawRow<__nv_bfloat16, kVec, kPairs> {
    using C = Columns<kVec, kPairs>;
    using V = Values<kPairs>;
    uint32_t w[kPairs];
    static constexpr int kWords = kPairs / 4;  // of 16 bytes
    __device__ __forceinline__ void take(const uint4* from, int step) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            const uint4 a = from[k * step];
            w[4 * k] = a.x, w[4 * k + 1] = a.y, w[4 * k + 2] = a.z, w[4 * k + 3] = a.w;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) w[k] = 0;
    }
    __device__ __forceinline__ void load(const char* at, const C& c) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(at);
        if constexpr (kVec && kPairs == 4) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else if constexpr (kVec) {
            const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p));
            w[0] = a.x, w[1] = a.y;
        } else {
            uint32_t half[C::kPer]{};
            c.each([&](int k) { half[k] = p[k * C::kStep]; });
#pragma unroll
            for (int k = 0; k < kPairs; ++k) w[k] = half[2 * k] | half[2 * k + 1] << 16;
        }
    }
    __device__ __forceinline__ V get() const {
        V r;
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
            r.v[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
        return r;
    }
    __device__ static __forceinline__ void store(char* at, const V& f, const C& c) {
        if (c.n == 0) return;
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(at);
        if (kVec) {
            uint32_t h[kPairs];
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f.v[k].x, f.v[k].y);
                h[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            if constexpr (kPairs == 4)
                *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
            else
                *reinterpret_cast<uint2*>(p) = make_uint2(h[0], h[1]);
        } else {
            const float* v = &f.v[0].x;
            c.each([&](int k) { p[k * C::kStep] = __float2bfloat16_rn(v[k]); });
        }
    }
};

// Means over the row: across lanes, then over the row's warps in order.  Two buffers in turn, so that
// one barrier is enough: who writes a buffer again has passed the barrier behind which all had read
// it.
struct RowSum {
    float4 (*buffer)[kMostThreads / 32];
    int turn, warps;
    float inv_width;

    __device__ __forceinline__ float4 over_warps(bool writes, float v, int at) {
        float4* to = buffer[turn];
        turn ^= 1;
        if (writes) (&to[threadIdx.x >> 5].x)[at] = v;
        __syncthreads();
        float4 s = to[0];
        // (Sums of up to four warps written out: 49.5 and 78.7 instead of 50.6 and 79.5 us at 32,400 x
        // 1,024, but 75.7 instead of 74.3 at 64,800 x 512 and 57.4 instead of 55.6 at 8,100 x 2,048 fp32.)
        for (int w = 1; w < warps; ++w) {
            const float4 o = to[w];
            s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
        }
        return s;
    }
    __device__ __forceinline__ float mean(float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (warps > 1) v = over_warps((threadIdx.x & 31) == 0, v, 0).x;
        return v * inv_width;
    }
    // Of four values: the halves of the warp take two of them each, their halves one: six steps
    // across lanes instead of twenty.
    __device__ __forceinline__ float4 mean(float a, float b, float c, float d) {
        const unsigned all = 0xffffffffu;
        const int lane = threadIdx.x & 31;
        const bool upper = lane & 16, odd = lane & 8;
        const float p = (upper ? c : a) + __shfl_xor_sync(all, upper ? a : c, 16);
        const float q = (upper ? d : b) + __shfl_xor_sync(all, upper ? b : d, 16);
        float v = (odd ? q : p) + __shfl_xor_sync(all, odd ? p : q, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(all, v, o);
        float4 s;
        if (warps > 1)
            s = over_warps((lane & 7) == 0, v, lane >> 3);
        else
            s = make_float4(__shfl_sync(all, v, 0), __shfl_sync(all, v, 8), __shfl_sync(all, v, 16),
                            __shfl_sync(all, v, 24));
        return make_float4(s.x * inv_width, s.y * inv_width, s.z * inv_width, s.w * inv_width);
    }
};

// the values less their mean m (layer norms), zero where there is none
template <bool kVec, int kPairs>
__device__ __forceinline__ void centre(Values<kPairs>& a, const Columns<kVec, kPairs>& c, float m) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) a.v[k] = add(a.v[k], both(-m));
    c.trim(a);
}

// The rows of block k of `blocks`, and the sequence of a token: consecutive.
__host__ __device__ __forceinline__ int64_t first_row(int64_t tokens, int64_t blocks, int64_t k) {
    return tokens * k / blocks;
}

struct Part {
    int b;               // sequence, -1: none holds the token
    int64_t begin, end;  // its tokens
};

__device__ __forceinline__ int64_t offset(const RnParams& p, int b) {
    return min64(max64(__ldg(p.cu + b), 0), p.tokens);
}

__device__ __forceinline__ Part part_of(const RnParams& p, int64_t t) {
    if (!p.cu) return {0, 0, p.tokens};
    int lo = 0, hi = p.batch + 1;  // the last offset at the token or before it
    if (offset(p, 0) > t) return {-1, 0, offset(p, 0)};
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offset(p, mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    if (lo == p.batch) return {-1, offset(p, lo), p.tokens};
    return {lo, offset(p, lo), offset(p, lo + 1)};
}

// Rows on their way to a thread: its words of the next kAhead rows of kArrays arrays, in shared memory.
// Each thread copies and takes its own words, so nothing but its own copies is waited for.  One row
// ahead in registers, as elsewhere, does not cover memory's latency where few blocks of large rows
// are on an SM: backward (16 warps), 32,400 x 1,024 in bfloat16 took 88.4 us that way and takes 79.5
// with 3 rows, 81.5 with 2, 80.3 with 4; forward, 8,100 x 4,096 58 and 49, but 64 x 256 4.1 and 4.5:
// there rows of up to 1,024 values have no ring.  In fp32, twice the words: 16,200 x 1,024, backward, 71 us
// without and 85 with it.
constexpr int kAhead = 3;
constexpr int kShortRow = 128;  // threads
template <typename T, bool kVec, int kThreads>
constexpr bool kUsesRing = kVec && sizeof(T) == 2 && kThreads > kShortRow;
template <typename Row, int kArrays>
struct RowRing {
    static constexpr int kRowWords = kArrays * Row::kWords;
    uint4* at;  // the thread's first word
    int step;   // words of the block's threads
    int stage;  // of the row that is next to be taken
    static size_t bytes(int threads) { return (size_t)kAhead * kRowWords * threads * 16; }
    __device__ __forceinline__ uint4* words(int s, int array) const {
        return at + (s * kRowWords + array * Row::kWords) * step;
    }
    __device__ __forceinline__ void bring(int s, int array, const char* from) const {
#pragma unroll
        for (int k = 0; k < Row::kWords; ++k) cp_async16(words(s, array) + k * step, from + k * 16);
    }
    __device__ __forceinline__ void take(Row& r, int array) const { r.take(words(stage, array), step); }
    __device__ __forceinline__ void next() { stage = stage == kAhead - 1 ? 0 : stage + 1; }
};

// beta gate times post's weight and bias, of sequence b (the first one's where none holds the row)
template <bool kVec, int kPairs>
__device__ __forceinline__ void mix_of(const RnParams& p, const Columns<kVec, kPairs>& c, int b,
                                       Values<kPairs>* factor, Values<kPairs>* rest) {
    const Values<kPairs> g =
        c.weights(p.gate ? p.gate + (int64_t)max(b, 0) * p.width : nullptr, 1.f);
    const Values<kPairs> w = c.weights(p.qw, 1.f);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) factor->v[k] = mul(mul(both(p.beta), g.v[k]), w.v[k]);
    if (!rest) return;
    const Values<kPairs> bias = c.weights(p.qb, 0.f);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) rest->v[k] = mul(mul(both(p.beta), g.v[k]), bias.v[k]);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// kLayer: one of the norms is a layer norm.  The statistics of the next row's y are formed with sums of
// this row, where there are such (ahead).
template <typename T, bool kVec, int kPairs, bool kLayer, bool kBias, int kThreads>
__global__ void __launch_bounds__(kThreads, kFwdWarps * 32 / kThreads) residual_norm_kernel(const RnParams p) {
    grid_dep_sync();
    using V = Values<kPairs>;
    using Row = RawRow<T, kVec, kPairs>;
    __shared__ float4 buffer[2][kMostThreads / 32];
    RowSum sums{buffer, 0, (int)blockDim.x / 32, 1.f / (float)p.width};
    const Columns<kVec, kPairs> c(p.width);
    const int64_t end = first_row(p.tokens, gridDim.x, blockIdx.x + 1);
    int64_t t = first_row(p.tokens, gridDim.x, blockIdx.x);
    Part at{0, 0, 0};
    // pre's weight and bias; the factor and the rest of un in r, those of the row's sequence
    const V pw = c.weights(p.pw, 1.f);
    V pb{}, factor{}, rest{};
    if (kBias) pb = c.weights(p.pb, 0.f);
    const int shift = c.first * (int)sizeof(T);
    Row x, y;
    x.clear();
    y.clear();
    const auto load = [&](uint32_t row) {
        if (c.n == 0) return;
        x.load(p.x.at(row, shift), c);
        if (p.y.p) y.load(p.y.at(row, shift), c);
    };
    constexpr bool kRing = kUsesRing<T, kVec, kThreads>;
    extern __shared__ uint4 ring_words[];
    RowRing<Row, 2> ring{ring_words + threadIdx.x, (int)blockDim.x, 0};
    const auto bring = [&](int stage, int64_t row) {
        if (kRing && c.n > 0 && row < end) {
            ring.bring(stage, 0, p.x.at((uint32_t)row, shift));
            if (p.y.p) ring.bring(stage, 1, p.y.at((uint32_t)row, shift));
        }
        cp_async_commit();
    };
    const auto take_y = [&]() {  // once its row is there: all but the two last ones that were brought
        cp_async_wait<kAhead - 1>();
        if constexpr (kRing)
            if (c.n > 0 && p.y.p) ring.take(y, 1);
    };
    if constexpr (kRing) {
        for (int s = 0; s < kAhead; ++s) bring(s, t + s);
        take_y();
    } else {
        load((uint32_t)t);
    }
    const bool centred = kLayer && p.post == GS_NORM_LAYER, centred_r = kLayer && p.pre == GS_NORM_LAYER;
    const bool ahead = p.post != GS_NORM_NONE && p.pre != GS_NORM_NONE && (!centred || centred_r);
    float mean_y = 0.f, square = 0.f;  // of y and, less its mean (layer norms), of y^2
    const auto statistics = [&](V u) {
        if (centred) {
            mean_y = sums.mean(total(u));
            centre(u, c, mean_y);
        }
        square = sums.mean(dot(u, u));
    };
    if (ahead) statistics(y.get());
    for (; t < end; ++t) {
        if constexpr (kRing)
            if (c.n > 0) ring.take(x, 0);
        V v = x.get(), u = y.get();
        if constexpr (kRing) {
            const int stage = ring.stage;
            ring.next();
            bring(stage, t + kAhead);
            take_y();
        } else if (t + 1 < end) {
            load((uint32_t)t + 1);
        }
        if (t >= at.end) {
            at = part_of(p, t);
            mix_of(p, c, at.b, &factor, kBias ? &rest : nullptr);
        }
        if (p.post != GS_NORM_NONE) {
            if (!ahead) statistics(u);
            if (centred) centre(u, c, mean_y);
            const float2 f = both(rsqrtf(square + p.eps));
#pragma unroll
            for (int k = 0; k < kPairs; ++k) u.v[k] = mul(u.v[k], f);
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
            v.v[k] = fma2(both(p.alpha), v.v[k],
                          kBias ? fma2(u.v[k], factor.v[k], rest.v[k]) : mul(u.v[k], factor.v[k]));
        if (p.r.p && at.b >= 0) Row::store(p.r.at((uint32_t)t, shift), v, c);
        if (p.pre == GS_NORM_NONE) continue;
        c.trim(v);
        float s;
        if (ahead) {
            V next = y.get();
            if (centred_r) {
                const float4 m = sums.mean(total(v), centred ? total(next) : 0.f, 0.f, 0.f);
                centre(v, c, m.x);
                if (centred) centre(next, c, mean_y = m.y);
            }
            const float4 m = sums.mean(dot(v, v), dot(next, next), 0.f, 0.f);
            s = m.x;
            square = m.y;
        } else {
            if (centred_r) centre(v, c, sums.mean(total(v)));
            s = sums.mean(dot(v, v));
        }
        const float2 f = both(rsqrtf(s + p.eps));
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
            v.v[k] = kBias ? fma2(mul(v.v[k], f), pw.v[k], pb.v[k]) : mul(mul(v.v[k], f), pw.v[k]);
        if (at.b >= 0) Row::store(p.h.at((uint32_t)t, shift), v, c);
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// The sums of dR un and of dR over rows of one sequence share the gate: kept without it, they give
// the gate's gradient and, with it, those of post's weight and bias.  kBias: there are biases or
// their gradients are wanted.  kLayer as above.
template <typename T, bool kVec, int kPairs, bool kLayer, bool kBias, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) residual_norm_bwd_kernel(const RnParams p) {
    grid_dep_sync();
    using V = Values<kPairs>;
    using Row = RawRow<T, kVec, kPairs>;
    __shared__ float4 buffer[2][kMostThreads / 32];
    RowSum sums{buffer, 0, (int)blockDim.x / 32, 1.f / (float)p.width};
    const Columns<kVec, kPairs> c(p.width);
    const int64_t begin = first_row(p.tokens, gridDim.x, blockIdx.x);
    const int64_t end = first_row(p.tokens, gridDim.x, blockIdx.x + 1);
    int64_t t = begin;
    Part at{-1, 0, 0};
    V dpw{}, dpb{}, dqw{}, dqb{};  // over all rows
    V su{}, s1{};                  // of dR un and of dR over the sequence's rows
    // pre's weight; the factor and the rest of un in r, those of the row's sequence
    const V pw = c.weights(p.pw, 1.f);
    V factor{}, rest{};
    const int shift = c.first * (int)sizeof(T);
    Row x, y, dr, dh;
    x.clear();
    y.clear();
    dr.clear();
    dh.clear();
    const auto load = [&](uint32_t row) {
        if (c.n == 0) return;
        x.load(p.x.at(row, shift), c);
        if (p.y.p) y.load(p.y.at(row, shift), c);
        if (p.dr.p) dr.load(p.dr.at(row, shift), c);
        if (p.dh.p) dh.load(p.dh.at(row, shift), c);
    };
    constexpr bool kRing = kUsesRing<T, kVec, kThreads>;
    extern __shared__ uint4 ring_words[];
    RowRing<Row, 4> ring{ring_words + threadIdx.x, (int)blockDim.x, 0};
    const auto bring = [&](int stage, int64_t row) {
        if (c.n > 0 && row < end) {
            const uint32_t at = (uint32_t)row;
            ring.bring(stage, 0, p.x.at(at, shift));
            if (p.y.p) ring.bring(stage, 1, p.y.at(at, shift));
            if (p.dr.p) ring.bring(stage, 2, p.dr.at(at, shift));
            if (p.dh.p) ring.bring(stage, 3, p.dh.at(at, shift));
        }
        cp_async_commit();
    };
    const auto take_y = [&]() {  // once its row is there: all but the two last ones that were brought
        cp_async_wait<kAhead - 1>();
        if constexpr (kRing)
            if (c.n > 0 && p.y.p) ring.take(y, 1);
    };
    // the sequence's sums to those of all rows, and to its gate's gradient
    const auto leave = [&]() {
        if (at.b < 0) return;
        V g = c.weights(p.gate ? p.gate + (int64_t)at.b * p.width : nullptr, 1.f);
        const V a = c.weights(p.qw, 1.f);
        V b{}, d;
        if (kBias) b = c.weights(p.qb, 0.f);
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            g.v[k] = mul(both(p.beta), g.v[k]);
            dqw.v[k] = fma2(g.v[k], su.v[k], dqw.v[k]);
            d.v[k] = mul(a.v[k], su.v[k]);
            if (kBias) {
                dqb.v[k] = fma2(g.v[k], s1.v[k], dqb.v[k]);
                d.v[k] = fma2(b.v[k], s1.v[k], d.v[k]);
                s1.v[k] = both(0.f);
            }
            d.v[k] = mul(both(p.beta), d.v[k]);
            su.v[k] = both(0.f);
        }
        if (!p.dgate) return;
        const bool from_before = at.begin < begin, goes_on = at.end > end;
        if (!from_before && !goes_on)
            c.store(p.dgate + (int64_t)at.b * p.width, d);
        else
            c.store(p.part_gate + ((int64_t)blockIdx.x * 2 + (from_before ? 0 : 1)) * p.width, d);
    };
    if constexpr (kRing) {
        for (int s = 0; s < kAhead; ++s) bring(s, t + s);
        take_y();
    } else {
        load((uint32_t)t);
    }
    const bool centred = kLayer && p.post == GS_NORM_LAYER;
    const bool ahead = p.post != GS_NORM_NONE && (!centred || p.pre != GS_NORM_NONE);
    float mean_y = 0.f, square = 0.f;  // of y and, less its mean (layer norms), of y^2
    const auto statistics = [&](V u) {
        if (centred) {
            mean_y = sums.mean(total(u));
            centre(u, c, mean_y);
        }
        square = sums.mean(dot(u, u));
    };
    if (ahead) statistics(y.get());
    for (; t < end; ++t) {
        if constexpr (kRing) {
            if (c.n > 0) {
                ring.take(x, 0);
                if (p.dr.p) ring.take(dr, 2);
                if (p.dh.p) ring.take(dh, 3);
            }
        }
        V v = x.get(), u = y.get(), d = dr.get();
        const V g = dh.get();
        if constexpr (kRing) {
            const int stage = ring.stage;
            ring.next();
            bring(stage, t + kAhead);
            take_y();
        } else if (t + 1 < end) {
            load((uint32_t)t + 1);
        }
        if (t >= at.end) {
            leave();
            at = part_of(p, t);
            mix_of(p, c, at.b, &factor, kBias ? &rest : nullptr);
        }
        // a row that no sequence holds is gone through like the others, but for the results
        const bool held = at.b >= 0;
        float fu = 1.f;
        if (p.post != GS_NORM_NONE) {
            if (!ahead) statistics(u);
            if (centred) centre(u, c, mean_y);
            fu = rsqrtf(square + p.eps);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) u.v[k] = mul(u.v[k], both(fu));  // un
        }
        if (p.pre != GS_NORM_NONE) {
#pragma unroll
            for (int k = 0; k < kPairs; ++k)
                v.v[k] = fma2(both(p.alpha), v.v[k],
                              kBias ? fma2(u.v[k], factor.v[k], rest.v[k])
                                    : mul(u.v[k], factor.v[k]));
            c.trim(v);
            if (kLayer && p.pre == GS_NORM_LAYER) centre(v, c, sums.mean(total(v)));
            V w;
#pragma unroll
            for (int k = 0; k < kPairs; ++k) w.v[k] = mul(pw.v[k], g.v[k]);
            const float4 s = sums.mean(dot(v, v), dot(w, v), kLayer ? total(w) : 0.f,
                                       centred ? total(y.get()) : 0.f);
            if (centred) mean_y = s.w;  // the next row's
            const float f = rsqrtf(s.x + p.eps);
            const float2 f2 = both(f), along = both(-s.y * f * f);
            const float2 mean = both(kLayer && p.pre == GS_NORM_LAYER ? -s.z : 0.f);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                if (held) {
                    dpw.v[k] = fma2(g.v[k], mul(v.v[k], f2), dpw.v[k]);
                    if (kBias) dpb.v[k] = add(dpb.v[k], g.v[k]);
                }
                if (kLayer) w.v[k] = add(w.v[k], mean);
                d.v[k] = fma2(f2, fma2(v.v[k], along, w.v[k]), d.v[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) v.v[k] = mul(both(p.alpha), d.v[k]);
        if (held) Row::store(p.dx.at((uint32_t)t, shift), v, c);
        if (!p.y.p) continue;
        if (held)
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                su.v[k] = fma2(d.v[k], u.v[k], su.v[k]);
                if (kBias) s1.v[k] = add(s1.v[k], d.v[k]);
            }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) d.v[k] = mul(d.v[k], factor.v[k]);
        if (p.post != GS_NORM_NONE) {
            c.trim(d);
            float4 s;
            if (ahead) {
                V next = y.get();
                if (centred) centre(next, c, mean_y);
                s = sums.mean(dot(d, u), dot(next, next), kLayer ? total(d) : 0.f, 0.f);
                square = s.y;
            } else {
                s = sums.mean(dot(d, u), 0.f, total(d), 0.f);
            }
            const float2 along = both(-s.x), mean = both(centred ? -s.z : 0.f);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                if (kLayer) d.v[k] = add(d.v[k], mean);
                d.v[k] = mul(both(fu), fma2(u.v[k], along, d.v[k]));
            }
        }
        if (held) Row::store(p.dy.at((uint32_t)t, shift), d, c);
    }
    leave();
    float* part = p.part + (int64_t)blockIdx.x * 4 * p.width;
    c.store(part, dpw);
    if (kBias) c.store(part + p.width, dpb);
    c.store(part + 2 * p.width, dqw);
    if (kBias) c.store(part + 3 * p.width, dqb);
}

// The blocks' sums of a column: 32 threads take every 32nd block, and their sums are added in
// pairs.  blockIdx.y: which of the four gradients, or behind them a sequence's gate (and every
// gridDim.y - 4 th from it on): of those that several blocks met, and zeros for empty ones.
constexpr int kFinishCols = 32, kFinishThreads = 1024, kFinishOf = kFinishThreads / kFinishCols;
constexpr int kFinishLoads = 10;  // of a thread at once: two rounds for 608 blocks
struct FourGradients {
    float* g[4];
};

__device__ __forceinline__ void sum_blocks(float (*s)[kFinishCols], const float* part, int first,
                                           int count, int64_t step, bool has, float* out) {
    const int col = threadIdx.x % kFinishCols, row = threadIdx.x / kFinishCols;
    float a = 0.f;
    if (has)
        for (int b0 = row; b0 < count; b0 += kFinishLoads * kFinishOf) {
            float v[kFinishLoads];
#pragma unroll
            for (int k = 0; k < kFinishLoads; ++k) {
                const int b = b0 + k * kFinishOf;
                v[k] = b < count ? __ldg(part + (first + b) * step) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kFinishLoads; ++k) a += v[k];
        }
    s[row][col] = a;
#pragma unroll
    for (int o = kFinishOf / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (row < o) s[row][col] += s[row + o][col];
    }
    if (row == 0 && has) *out = s[0][col];
}

__global__ void __launch_bounds__(kFinishThreads)
    residual_norm_finish_kernel(const RnParams p, int blocks, FourGradients out) {
    grid_dep_sync();
    __shared__ float s[kFinishOf][kFinishCols];
    const int col = blockIdx.x * kFinishCols + threadIdx.x % kFinishCols;
    const bool has = col < p.width;
    if (blockIdx.y < 4) {
        float* to = out.g[blockIdx.y];
        if (to)
            sum_blocks(s, p.part + (int64_t)blockIdx.y * p.width + col, 0, blocks, 4 * (int64_t)p.width,
                       has, to + col);
        return;
    }
    const int64_t w = p.width;
    for (int b = blockIdx.y - 4; b < p.batch; b += gridDim.y - 4) {
        const int64_t begin = p.cu ? offset(p, b) : 0, end = p.cu ? offset(p, b + 1) : p.tokens;
        float* to = p.dgate + b * w + col;
        if (end <= begin) {
            if (has && threadIdx.x < kFinishCols) *to = 0.f;
            continue;
        }
        const auto block_of = [&](int64_t t) {
            int64_t k = t * blocks / p.tokens;  // or one off
            while (k + 1 < blocks && first_row(p.tokens, blocks, k + 1) <= t) ++k;
            while (k > 0 && first_row(p.tokens, blocks, k) > t) --k;
            return (int)k;
        };
        const int first = block_of(begin), last = block_of(end - 1);
        if (first == last) continue;  // the block has written it
        // The first block keeps it as its last sequence: in the second of its places, unless it
        // began before the block, which only offsets out of order make it; the others in the first.
        __syncthreads();
        const float* part = p.part_gate + col;
        const bool here = first_row(p.tokens, blocks, first) <= begin;
        if (threadIdx.x < kFinishCols && has)
            s[0][threadIdx.x] = __ldg(part + ((int64_t)first * 2 + (here ? 1 : 0)) * w);
        __syncthreads();
        const float head = s[0][threadIdx.x % kFinishCols];
        __syncthreads();
        sum_blocks(s, part, first + 1, last - first, 2 * w, has, to);
        if (threadIdx.x < kFinishCols && has) *to += head;
    }
}

// How a row is shared out: threads of eight values, or of four where their addresses and column
// sums would not fit the registers: odd widths in fp32 with biases or a layer norm.  (With both,
// backward and forward, with four values: 16,200 x 515 77 and 40 us, 16,200 x 1,001 124 and 61, 8,103 x
// 2,047 151 and 73; with eight 120 and 41, 180 and 60, 200 and 65.  Without either, 16,200 x 1,001: 78
// with four and 66 with eight; 32,400 x 1,001 in bfloat16 377 and 199.  96 registers, for five rows
// instead of four at 515 values: 34 us instead of 31 on 4,346.)
int pairs_of(const RnParams& p, bool vec, bool bf16, bool bias) {
    const bool layer = p.pre == GS_NORM_LAYER || p.post == GS_NORM_LAYER;
    return !vec && !bf16 && (bias || layer) && p.width <= kFourUpTo ? 2 : 4;
}

int warps_of(int width, int pairs) { return (width + 64 * pairs - 1) / (64 * pairs); }

int64_t most_blocks(int width, int pairs, int resident_warps) {
    return (int64_t)kSms * std::max(1, resident_warps / warps_of(width, pairs));
}

NormRows rows_of(const gs_rows& r, int size) {
    return {static_cast<char*>(r.data), (uint32_t)(r.row_stride * size)};
}

RnParams params_of(const ResidualNormArgs& a, const gs_rows& x, const gs_rows& y) {
    RnParams p{};
    const int size = a.bf16 ? 2 : 4;
    p.tokens = a.tokens;
    p.width = a.width;
    p.batch = a.batch;
    p.pre = a.pre;
    p.post = a.post;
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.eps = a.eps;
    p.pw = a.w.pre_weight;
    p.pb = a.w.pre_bias;
    p.qw = a.w.post_weight;
    p.qb = a.w.post_bias;
    p.gate = a.w.gate;
    p.cu = a.cu;
    p.x = rows_of(x, size);
    p.y = rows_of(y, size);
    return p;
}

// whole 16-byte words: a thread's values lie side by side (of weights and gates too)
bool whole_words(int width, std::initializer_list<NormRows> arrays) {
    if (width % 8) return false;
    for (const NormRows& r : arrays)
        if (reinterpret_cast<uintptr_t>(r.p) % 16 || (r.p && r.stride % 16)) return false;
    return true;
}

// With the shared memory of a ring for kArrays arrays.  The kernel's limit on it is that of the widest
// row, whatever this call's width: it belongs to the kernel, and another thread's call may set it
// between this one's setting and launch.
template <typename T, bool kVec, int kPairs, int kThreads, int kArrays>
cudaError_t launch_rows(void (*kernel)(const RnParams), const RnParams& p, unsigned blocks,
                        cudaStream_t st) {
    const unsigned threads = (unsigned)warps_of(p.width, kPairs) * 32;
    size_t ring = 0;
    if constexpr (kUsesRing<T, kVec, kThreads>) {
        using Ring = RowRing<RawRow<T, kVec, kPairs>, kArrays>;
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Ring::bytes(kThreads));
        if (e != cudaSuccess) return e;
        ring = Ring::bytes(threads);
    }
    return launch(kernel, dim3(blocks), dim3(threads), ring, st, p);
}

template <typename T, bool kVec, int kPairs, int kThreads>
cudaError_t launch_fwd_of(const RnParams& p, bool bias, cudaStream_t st) {
    const bool layer = p.pre == GS_NORM_LAYER || p.post == GS_NORM_LAYER;
    void (*kernel)(const RnParams);
    if (layer)
        kernel = bias ? residual_norm_kernel<T, kVec, kPairs, true, true, kThreads>
                      : residual_norm_kernel<T, kVec, kPairs, true, false, kThreads>;
    else
        kernel = bias ? residual_norm_kernel<T, kVec, kPairs, false, true, kThreads>
                      : residual_norm_kernel<T, kVec, kPairs, false, false, kThreads>;
    return launch_rows<T, kVec, kPairs, kThreads, 2>(
        kernel, p, (unsigned)std::min(p.tokens, most_blocks(p.width, kPairs, kFwdWarps)), st);
}

template <typename T, bool kVec>
cudaError_t launch_fwd(const RnParams& p, cudaStream_t st) {
    const bool bias = p.pb || p.qb;
    if constexpr (!kVec && sizeof(T) == 4)
        if (pairs_of(p, kVec, false, bias) == 2)
            return launch_fwd_of<T, kVec, 2, 512>(p, bias, st);
    if constexpr (kVec && sizeof(T) == 2)
        if (warps_of(p.width, 4) * 32 <= kShortRow)
            return launch_fwd_of<T, kVec, 4, kShortRow>(p, bias, st);
    return launch_fwd_of<T, kVec, 4, kMostThreads>(p, bias, st);
}

template <typename T, bool kVec, int kPairs, int kThreads>
cudaError_t launch_bwd_of(const RnParams& p, bool bias, int blocks, cudaStream_t st) {
    const bool layer = p.pre == GS_NORM_LAYER || p.post == GS_NORM_LAYER;
    void (*kernel)(const RnParams);
    if (layer)
        kernel = bias ? residual_norm_bwd_kernel<T, kVec, kPairs, true, true, kThreads>
                      : residual_norm_bwd_kernel<T, kVec, kPairs, true, false, kThreads>;
    else
        kernel = bias ? residual_norm_bwd_kernel<T, kVec, kPairs, false, true, kThreads>
                      : residual_norm_bwd_kernel<T, kVec, kPairs, false, false, kThreads>;
    return launch_rows<T, kVec, kPairs, kThreads, 4>(kernel, p, (unsigned)blocks, st);
}

// Up to 4,096 values a row its threads may have 128 registers each; beyond, 64 and spills.  (Without
// a number of blocks in its bounds the compiler gave these 32: 577 us instead of 268 on 2,025 x 8,192 in
// fp32.)
template <typename T, bool kVec>
cudaError_t launch_bwd(const RnParams& p, bool bias, int blocks, cudaStream_t st) {
    if constexpr (!kVec && sizeof(T) == 4)
        if (pairs_of(p, kVec, false, bias) == 2)
            return launch_bwd_of<T, kVec, 2, 512>(p, bias, blocks, st);
    if (warps_of(p.width, 4) <= 16) return launch_bwd_of<T, kVec, 4, 512>(p, bias, blocks, st);
    return launch_rows<T, kVec, 4, kMostThreads, 4>(
        residual_norm_bwd_kernel<T, kVec, 4, true, true, kMostThreads>, p, (unsigned)blocks, st);
}

}  // namespace

size_t residual_norm_workspace_bytes(int width) {
    const int64_t blocks = most_blocks(width, 4, kBwdWarps);  // with fewer values a thread: fewer
    return (size_t)blocks * 6 * width * sizeof(float) + 16;
}

cudaError_t launch_residual_norm(const ResidualNormArgs& a, const gs_rows& x, const gs_rows& y,
                                 const gs_rows& r, const gs_rows& h, cudaStream_t st) {
    RnParams p = params_of(a, x, y);
    const int size = a.bf16 ? 2 : 4;
    p.r = rows_of(r, size);
    p.h = rows_of(h, size);
    const bool vec = whole_words(a.width, {p.x, p.y, p.r, p.h});
    if (a.bf16)
        return vec ? launch_fwd<__nv_bfloat16, true>(p, st) : launch_fwd<__nv_bfloat16, false>(p, st);
    return vec ? launch_fwd<float, true>(p, st) : launch_fwd<float, false>(p, st);
}

cudaError_t launch_residual_norm_bwd(const ResidualNormArgs& a, const gs_rows& x, const gs_rows& y,
                                     const gs_rows& dr, const gs_rows& dh, const gs_rows& dx,
                                     const gs_rows& dy, const gs_norm_grads& g, void* ws,
                                     cudaStream_t st) {
    RnParams p = params_of(a, x, y);
    const int size = a.bf16 ? 2 : 4;
    p.dr = rows_of(dr, size);
    p.dh = rows_of(dh, size);
    p.dx = rows_of(dx, size);
    p.dy = rows_of(dy, size);
    p.dgate = g.gate;
    const bool vec = whole_words(a.width, {p.x, p.y, p.dr, p.dh, p.dx, p.dy});
    const bool bias = p.pb || p.qb || g.pre_bias || g.post_bias;
    const int pairs = pairs_of(p, vec, a.bf16, bias);
    const int blocks = (int)std::min(a.tokens, most_blocks(a.width, pairs, kBwdWarps));
    p.part = static_cast<float*>(ws);
    p.part_gate = p.part + ((int64_t)blocks * 4 * a.width + 3) / 4 * 4;
    cudaError_t e = cudaSuccess;
    if (a.tokens > 0 && a.bf16)
        e = vec ? launch_bwd<__nv_bfloat16, true>(p, bias, blocks, st)
                : launch_bwd<__nv_bfloat16, false>(p, bias, blocks, st);
    else if (a.tokens > 0)
        e = vec ? launch_bwd<float, true>(p, bias, blocks, st)
                : launch_bwd<float, false>(p, bias, blocks, st);
    const FourGradients out{{g.pre_weight, g.pre_bias, g.post_weight, g.post_bias}};
    const bool sums = g.pre_weight || g.pre_bias || g.post_weight || g.post_bias;
    if (e == cudaSuccess && (sums || g.gate))
        e = launch(residual_norm_finish_kernel,
                   dim3((unsigned)((a.width + kFinishCols - 1) / kFinishCols),
                        4u + (g.gate ? (unsigned)std::min(a.batch, kMostGates) : 0u)),
                   dim3(kFinishThreads), 0, st, p, blocks, out);
    return e;
}

}  // namespace gs
