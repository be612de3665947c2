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
// of at most 256 values is one warp's and its sums need no barrier.  Weights and gates come
// from L1 for every row: in registers they would take half of the warps' room.  A block has
// consecutive rows, reads the next one while it works on the present one, and keeps sums of the
// column gradients in registers: of the weights and biases over all its rows, of the gate over
// those of a sequence.  Other kernels add the blocks' sums up in the blocks' order: the same
// inputs give the same bits.
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
constexpr int kPer = 8;             // values a thread
constexpr int kMostThreads = 1024;  // width <= 8,192
constexpr int kFwdWarps = 32, kBwdWarps = 16;  // resident on an SM
constexpr int kSumThreads = 256;

struct NormRows {
    char* p;
    int64_t stride;  // bytes
    __device__ __forceinline__ char* row(int64_t t) const { return p + t * stride; }
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

// A thread's eight columns: neighbours, or (odd widths and strides) every blockDim-th.
template <bool kVec>
struct Columns {
    int first, step, n;  // n: those that exist
    __device__ __forceinline__ Columns(int width) {
        first = kVec ? (int)threadIdx.x * kPer : (int)threadIdx.x;
        step = kVec ? 1 : (int)blockDim.x;
        n = first >= width ? 0 : kVec ? kPer : min(kPer, (width - 1 - first) / step + 1);
    }
    __device__ __forceinline__ void weights(float (&v)[kPer], const float* w, float other) const {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = other;
        if (!w || n == 0) return;
        if (kVec) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(w + first));
            const float4 b = __ldg(reinterpret_cast<const float4*>(w + first) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (k < n) v[k] = __ldg(w + first + k * step);
        }
    }
    __device__ __forceinline__ void store(float* w, const float (&v)[kPer]) const {
        if (n == 0) return;
        if (kVec) {
            reinterpret_cast<float4*>(w + first)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(w + first)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (k < n) w[first + k * step] = v[k];
        }
    }
};

// A thread's values of a row as they lie in memory, zeros where there is none.
template <typename T, bool kVec>
struct RawRow;

template <bool kVec>
struct RawRow<float, kVec> {
    float v[kPer];
    __device__ __forceinline__ void load(const char* row, const Columns<kVec>& c) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = 0.f;
        if (!row || c.n == 0) return;
        const float* p = reinterpret_cast<const float*>(row) + c.first;
        if (kVec) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
            const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (k < c.n) v[k] = p[k * c.step];
        }
    }
    __device__ __forceinline__ void get(float (&f)[kPer]) const {
#pragma unroll
        for (int k = 0; k < kPer; ++k) f[k] = v[k];
    }
    __device__ static __forceinline__ void store(char* row, const float (&f)[kPer],
                                                 const Columns<kVec>& c) {
        c.store(reinterpret_cast<float*>(row), f);
    }
};

template <bool kVec>
struct RawRow<__nv_bfloat16, kVec> {
    uint32_t w[kPer / 2];
    __device__ __forceinline__ void load(const char* row, const Columns<kVec>& c) {
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) w[k] = 0;
        if (!row || c.n == 0) return;
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + c.first;
        if (kVec) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (k < c.n) w[k / 2] |= (uint32_t)p[k * c.step] << (16 * (k & 1));
        }
    }
    __device__ __forceinline__ void get(float (&f)[kPer]) const {
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) {
            f[2 * k] = __uint_as_float(w[k] << 16);
            f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    __device__ static __forceinline__ void store(char* row, const float (&f)[kPer],
                                                 const Columns<kVec>& c) {
        if (c.n == 0) return;
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(row) + c.first;
        if (kVec) {
            __nv_bfloat162 h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (k < c.n) p[k * c.step] = __float2bfloat16_rn(f[k]);
        }
    }
};

// Sums over the row: lanes, then the row's warps in order.  Two buffers in turn, so that one
// barrier a sum is enough: who writes a buffer again has passed the barrier behind which all had
// read it.
constexpr int kMostSums = 3;
struct RowSum {
    float (*buffer)[kMostSums][kMostThreads / 32];
    int turn, warps;
    float inv_width;

    template <int kN>
    __device__ __forceinline__ void mean(float (&v)[kN]) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if (warps > 1) {
            float(*to)[kMostThreads / 32] = buffer[turn];
            turn ^= 1;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int k = 0; k < kN; ++k) to[k][threadIdx.x >> 5] = v[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kN; ++k) v[k] = to[k][0];
            for (int w = 1; w < warps; ++w)
#pragma unroll
                for (int k = 0; k < kN; ++k) v[k] += to[k][w];
        }
#pragma unroll
        for (int k = 0; k < kN; ++k) v[k] *= inv_width;
    }
};

// the values less their mean (layer norms), zero where there is none
__device__ __forceinline__ void centre(float (&v)[kPer], int n, int kind, RowSum& sums) {
    if (kind != GS_NORM_LAYER) return;
    float m[1] = {0.f};
#pragma unroll
    for (int k = 0; k < kPer; ++k) m[0] += v[k];
    sums.mean(m);
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = k < n ? v[k] - m[0] : 0.f;
}

__device__ __forceinline__ float square_sum(const float (&v)[kPer]) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) s = fmaf(v[k], v[k], s);
    return s;
}

// values to those of the norm, without weight and bias; returns the factor
__device__ __forceinline__ float normalise(float (&v)[kPer], int n, int kind, float eps,
                                           RowSum& sums) {
    if (kind == GS_NORM_NONE) return 1.f;
    centre(v, n, kind, sums);
    float s[1] = {square_sum(v)};
    sums.mean(s);
    const float f = rsqrtf(s[0] + eps);
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] *= f;
    return f;
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

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename T, bool kVec>
__global__ void __launch_bounds__(kMostThreads) residual_norm_kernel(const RnParams p) {
    grid_dep_sync();
    __shared__ float buffer[2][kMostSums][kMostThreads / 32];
    RowSum sums{buffer, 0, (int)blockDim.x / 32, 1.f / (float)p.width};
    const Columns<kVec> c(p.width);
    const int64_t end = first_row(p.tokens, gridDim.x, blockIdx.x + 1);
    int64_t t = first_row(p.tokens, gridDim.x, blockIdx.x);
    Part at{0, 0, 0};
    RawRow<T, kVec> x, y;
    const auto load = [&](int64_t row) {
        x.load(row < end ? p.x.row(row) : nullptr, c);
        y.load(row < end && p.y.p ? p.y.row(row) : nullptr, c);
    };
    load(t);
    for (; t < end; ++t) {
        float v[kPer], u[kPer], w[kPer];
        x.get(v);
        y.get(u);
        load(t + 1);
        if (t >= at.end) at = part_of(p, t);
        if (at.b < 0) continue;
        normalise(u, c.n, p.post, p.eps, sums);
        c.weights(w, p.gate ? p.gate + (int64_t)at.b * p.width : nullptr, 1.f);
        float a[kPer], b[kPer];
        c.weights(a, p.qw, 1.f);
        c.weights(b, p.qb, 0.f);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            v[k] = fmaf(p.alpha, v[k], p.beta * w[k] * fmaf(u[k], a[k], b[k]));
        if (p.r.p) RawRow<T, kVec>::store(p.r.row(t), v, c);
        if (p.pre == GS_NORM_NONE) continue;
        normalise(v, c.n, p.pre, p.eps, sums);
        c.weights(a, p.pw, 1.f);
        c.weights(b, p.pb, 0.f);
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = fmaf(v[k], a[k], b[k]);
        RawRow<T, kVec>::store(p.h.row(t), v, c);
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// The sums of du un and of du over rows of one sequence share the gate: kept without it, they
// give the gate's gradient too.
template <typename T, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads) residual_norm_bwd_kernel(const RnParams p) {
    grid_dep_sync();
    __shared__ float buffer[2][kMostSums][kMostThreads / 32];
    RowSum sums{buffer, 0, (int)blockDim.x / 32, 1.f / (float)p.width};
    const Columns<kVec> c(p.width);
    const int64_t begin = first_row(p.tokens, gridDim.x, blockIdx.x);
    const int64_t end = first_row(p.tokens, gridDim.x, blockIdx.x + 1);
    int64_t t = begin;
    Part at{-1, 0, 0};
    float dpw[kPer]{}, dpb[kPer]{}, dqw[kPer]{}, dqb[kPer]{};  // over all rows
    float su[kPer]{}, s1[kPer]{};  // sums of dR un and of dR over the sequence's rows
    RawRow<T, kVec> x, y, dr, dh;
    const auto load = [&](int64_t row) {
        const bool some = row < end;
        x.load(some ? p.x.row(row) : nullptr, c);
        y.load(some && p.y.p ? p.y.row(row) : nullptr, c);
        dr.load(some && p.dr.p ? p.dr.row(row) : nullptr, c);
        dh.load(some && p.dh.p ? p.dh.row(row) : nullptr, c);
    };
    // the sequence's sums to those of all rows, and to its gate's gradient
    const auto leave = [&]() {
        if (at.b < 0) return;
        float g[kPer], a[kPer], b[kPer], d[kPer];
        c.weights(g, p.gate ? p.gate + (int64_t)at.b * p.width : nullptr, 1.f);
        c.weights(a, p.qw, 1.f);
        c.weights(b, p.qb, 0.f);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            dqw[k] = fmaf(p.beta * g[k], su[k], dqw[k]);
            dqb[k] = fmaf(p.beta * g[k], s1[k], dqb[k]);
            d[k] = p.beta * fmaf(a[k], su[k], b[k] * s1[k]);
            su[k] = s1[k] = 0.f;
        }
        if (!p.dgate) return;
        const bool from_before = at.begin < begin, goes_on = at.end > end;
        if (!from_before && !goes_on)
            c.store(p.dgate + (int64_t)at.b * p.width, d);
        else
            c.store(p.part_gate + ((int64_t)blockIdx.x * 2 + (from_before ? 0 : 1)) * p.width, d);
    };
    load(t);
    for (; t < end; ++t) {
        float v[kPer], u[kPer], g[kPer], w[kPer], d[kPer];
        x.get(v);
        y.get(u);
        dr.get(d);
        dh.get(g);
        load(t + 1);
        if (t >= at.end) {
            leave();
            at = part_of(p, t);
        }
        if (at.b < 0) continue;
        const float fu = normalise(u, c.n, p.post, p.eps, sums);  // un
        float bg[kPer], qw[kPer];
        c.weights(bg, p.gate ? p.gate + (int64_t)at.b * p.width : nullptr, 1.f);
        c.weights(qw, p.qw, 1.f);
#pragma unroll
        for (int k = 0; k < kPer; ++k) bg[k] *= p.beta;
        if (p.pre != GS_NORM_NONE) {
            c.weights(w, p.qb, 0.f);
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                v[k] = k < c.n ? fmaf(p.alpha, v[k], bg[k] * fmaf(u[k], qw[k], w[k])) : 0.f;
            centre(v, c.n, p.pre, sums);
            c.weights(w, p.pw, 1.f);
            float s[3] = {square_sum(v), 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                w[k] *= g[k];
                s[1] = fmaf(w[k], v[k], s[1]);
                s[2] += w[k];
            }
            sums.mean(s);
            const float f = rsqrtf(s[0] + p.eps), along = s[1] * f;
            const float mean = p.pre == GS_NORM_LAYER ? s[2] : 0.f;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const float vn = v[k] * f;
                dpw[k] = fmaf(g[k], vn, dpw[k]);
                dpb[k] += g[k];
                d[k] = fmaf(f, (w[k] - mean) - vn * along, d[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = p.alpha * d[k];
        RawRow<T, kVec>::store(p.dx.row(t), v, c);
        if (!p.y.p) continue;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            su[k] = fmaf(d[k], u[k], su[k]);
            s1[k] += d[k];
            d[k] *= bg[k];
        }
        if (p.post != GS_NORM_NONE) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                d[k] = k < c.n ? d[k] * qw[k] : 0.f;
                s[0] = fmaf(d[k], u[k], s[0]);
                s[1] += d[k];
            }
            sums.mean(s);
            const float mean = p.post == GS_NORM_LAYER ? s[1] : 0.f;
#pragma unroll
            for (int k = 0; k < kPer; ++k) d[k] = fu * ((d[k] - mean) - u[k] * s[0]);
        }
        RawRow<T, kVec>::store(p.dy.row(t), d, c);
    }
    leave();
    float* part = p.part + (int64_t)blockIdx.x * 4 * p.width;
    c.store(part, dpw);
    c.store(part + p.width, dpb);
    c.store(part + 2 * p.width, dqw);
    c.store(part + 3 * p.width, dqb);
}

// The blocks' sums of a column: 32 threads take every 32nd block, and their sums are added in
// order.  blockIdx.y: which of the four gradients.
constexpr int kFinishCols = 32, kFinishThreads = 1024;
struct FourGradients {
    float* g[4];
};
__global__ void __launch_bounds__(kFinishThreads)
    residual_norm_sum_kernel(const float* __restrict__ part, int blocks, int width,
                             FourGradients out) {
    grid_dep_sync();
    if (!out.g[blockIdx.y]) return;
    constexpr int kOf = kFinishThreads / kFinishCols;
    __shared__ float s[kOf][kFinishCols];
    const int col = threadIdx.x % kFinishCols, row = threadIdx.x / kFinishCols;
    const int i = blockIdx.x * kFinishCols + col;
    float a = 0.f;
    if (i < width)
#pragma unroll 8
        for (int b = row; b < blocks; b += kOf)
            a += __ldg(part + ((int64_t)b * 4 + blockIdx.y) * width + i);
    s[row][col] = a;
    __syncthreads();
    if (row != 0 || i >= width) return;
    for (int r = 1; r < kOf; ++r) a += s[r][col];
    out.g[blockIdx.y][i] = a;
}

// The gate's gradient of sequences that several blocks met, in the blocks' order, and of empty ones.
__global__ void __launch_bounds__(kSumThreads) residual_norm_gate_kernel(const RnParams p, int blocks) {
    grid_dep_sync();
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        const int64_t begin = p.cu ? offset(p, b) : 0, end = p.cu ? offset(p, b + 1) : p.tokens;
        const auto block_of = [&](int64_t t) {
            int64_t k = t * blocks / p.tokens;  // its first row may lie before t, or one block on
            while (k + 1 < blocks && first_row(p.tokens, blocks, k + 1) <= t) ++k;
            while (k > 0 && first_row(p.tokens, blocks, k) > t) --k;
            return (int)k;
        };
        const bool some = end > begin;
        const int first = some ? block_of(begin) : 0, last = some ? block_of(end - 1) : 0;
        if (some && first == last) continue;
        for (int i = blockIdx.y * kSumThreads + threadIdx.x; i < p.width; i += gridDim.y * kSumThreads) {
            float a = 0.f;
            if (some) {
                // the first block's last sequence -- unless it is its first one too
                const bool before = first_row(p.tokens, blocks, first) > begin;
                a = __ldg(p.part_gate + ((int64_t)first * 2 + (before ? 0 : 1)) * p.width + i);
#pragma unroll 8
                for (int k = first + 1; k <= last; ++k)
                    a += __ldg(p.part_gate + (int64_t)k * 2 * p.width + i);
            }
            p.dgate[(int64_t)b * p.width + i] = a;
        }
    }
}

int warps_of(int width) { return (width + 32 * kPer - 1) / (32 * kPer); }

int blocks_of(int64_t tokens, int width, int resident_warps) {
    return (int)std::min<int64_t>(tokens, (int64_t)kSms * std::max(1, resident_warps / warps_of(width)));
}

NormRows rows_of(const gs_rows& r, int size) {
    return {static_cast<char*>(r.data), r.row_stride * size};
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

// whole 16-byte words: eight values a thread lie side by side (rows of the weights too)
bool whole_words(int width, std::initializer_list<NormRows> arrays) {
    if (width % kPer) return false;
    for (const NormRows& r : arrays)
        if (reinterpret_cast<uintptr_t>(r.p) % 16 || (r.p && r.stride % 16)) return false;
    return true;
}

template <typename T, bool kVec>
cudaError_t launch_fwd(const RnParams& p, int blocks, cudaStream_t st) {
    return launch(residual_norm_kernel<T, kVec>, dim3((unsigned)blocks),
                  dim3((unsigned)warps_of(p.width) * 32), 0, st, p);
}

// Up to 4,096 values a row its threads may have 128 registers each; beyond, 64 and spills.
template <typename T, bool kVec>
cudaError_t launch_bwd(const RnParams& p, int blocks, cudaStream_t st) {
    const unsigned threads = (unsigned)warps_of(p.width) * 32;
    return launch(threads <= 512 ? residual_norm_bwd_kernel<T, kVec, 512>
                                 : residual_norm_bwd_kernel<T, kVec, kMostThreads>,
                  dim3((unsigned)blocks), dim3(threads), 0, st, p);
}

}  // namespace

size_t residual_norm_workspace_bytes(int width) {
    const size_t blocks = (size_t)kSms * std::max(1, kBwdWarps / warps_of(width));
    return blocks * 6 * width * sizeof(float) + 16;
}

cudaError_t launch_residual_norm(const ResidualNormArgs& a, const gs_rows& x, const gs_rows& y,
                                 const gs_rows& r, const gs_rows& h, cudaStream_t st) {
    RnParams p = params_of(a, x, y);
    const int size = a.bf16 ? 2 : 4;
    p.r = rows_of(r, size);
    p.h = rows_of(h, size);
    const bool vec = whole_words(a.width, {p.x, p.y, p.r, p.h});
    const int blocks = blocks_of(a.tokens, a.width, kFwdWarps);
    if (a.bf16)
        return vec ? launch_fwd<__nv_bfloat16, true>(p, blocks, st)
                   : launch_fwd<__nv_bfloat16, false>(p, blocks, st);
    return vec ? launch_fwd<float, true>(p, blocks, st) : launch_fwd<float, false>(p, blocks, st);
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
    const int blocks = blocks_of(a.tokens, a.width, kBwdWarps);
    p.part = static_cast<float*>(ws);
    p.part_gate = p.part + ((int64_t)blocks * 4 * a.width + 3) / 4 * 4;
    const bool vec = whole_words(a.width, {p.x, p.y, p.dr, p.dh, p.dx, p.dy});
    cudaError_t e = cudaSuccess;
    if (a.tokens > 0 && a.bf16)
        e = vec ? launch_bwd<__nv_bfloat16, true>(p, blocks, st)
                : launch_bwd<__nv_bfloat16, false>(p, blocks, st);
    else if (a.tokens > 0)
        e = vec ? launch_bwd<float, true>(p, blocks, st) : launch_bwd<float, false>(p, blocks, st);
    const FourGradients out{{g.pre_weight, g.pre_bias, g.post_weight, g.post_bias}};
    if (e == cudaSuccess && (g.pre_weight || g.pre_bias || g.post_weight || g.post_bias))
        e = launch(residual_norm_sum_kernel,
                   dim3((a.width + kFinishCols - 1) / kFinishCols, 4), dim3(kFinishThreads), 0, st,
                   (const float*)p.part, blocks, a.width, out);
    if (e == cudaSuccess && g.gate)
        e = launch(residual_norm_gate_kernel,
                   dim3((unsigned)std::min(a.batch, 4 * kSms),
                        (unsigned)((a.width + kSumThreads - 1) / kSumThreads)),
                   dim3(kSumThreads), 0, st, p, blocks);
    return e;
}

}  // namespace gs
