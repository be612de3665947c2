// gs_headnorm.cu -- RMS norm of every query and key head and the position
// rotation in one pass, and its gradient.
//
// A head's row x of D values becomes n = r w x with r = (mean x^2 + eps)^(-1/2);
// the first `rot` values of n are taken as rot/2 pairs (a, b) and turned by the
// token's angles: (a c - b s, b c + a s).  With a pair's weights w_a and w_b the
// outputs are r (a c w_a - b s w_b) and r (b c w_b + a s w_a), four factors that a
// token's rows share.  The gradient turns dy back by the same angles into g, and with
// s2 = sum x^2, t = sum_j w_j g_j x_j
//   dx_j = r (w_j g_j - x_j r^2 t / D),   dw_j = sum over rows of g_j x_j r,
// so one pass with two sums over the row serves it.
//
// Memory bounds it (about 14 operations for 6 bytes in bfloat16) as long as the
// instructions are few and the bytes in flight many.  A lane takes four pairs of a row
// -- both halves of each, so that no value crosses lanes but the two sums -- a row the
// next power of two of D / 8 lanes, and a warp kRows rows a lane of one token, all of
// whose loads it issues at once, the angles among them; the token's place in the table
// is read a token ahead.  Columns that are not rotated are taken in pairs too, with
// cosine 1 and sine 0.
//
// Two rows of bfloat16 a lane and four blocks an SM in the forward (32 warps, 64
// registers), three in the gradient: more rows a lane mean fewer warps, and 32,400
// tokens x (16 + 4) heads x 128 took 76 instead of 63 us with four rows and three
// blocks, 105 with one row and six.  A ring of asynchronous copies in shared memory was
// no faster (75 us): its bookkeeping took more issue slots than its depth hid.
// Measured there: 63 us forward (5.5 TB/s of the bytes it cannot do without, 0.83 of
// the copy rate), 107 us with the gradient's three arrays (4.8 TB/s, 0.72).
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
constexpr int kSms = 152;
constexpr int kFwdBlocks = 4 * kSms, kBwdBlocks = 3 * kSms;  // resident at once
constexpr int kFinishCols = 32, kFinishThreads = 1024;

// How the pairs lie: halves in whole groups of 4 pairs, halves otherwise, neighbours.  Halves
// whose columns no 4 pairs hold are read and written one by one: 32,400 tokens x (16 + 4) heads x
// 72 in bfloat16 take 126 us with 36 values rotated, 57 with all 72.
enum Pairing : int { kHalves4 = 0, kHalves = 1, kNeighbours = 2 };

struct Rows {
    char* p;
    int64_t ts, hs;  // strides in bytes
};

// parts of a token's heads, and warps that walk the tokens for each
struct Share {
    int parts, warps;
};

struct HnParams {
    int64_t tokens, table_rows;
    int hq, hk, dim, rot;
    Share share[4];  // full parts of the queries' heads, their last one; the keys' likewise
    float eps;
    const float *qw, *kw, *cos_sin;
    const int32_t* positions;
    Rows q, k, yq, yk;    // inputs; outputs (forward) or the outputs' gradients (backward)
    Rows dq, dk;          // backward
    float* part;          // backward: [blocks][2][dim]
};

// Four pairs of a row, as they lie in memory.
struct Four {  // the pairs' first values, then their second ones
    float2 a[2], b[2];
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <typename T>
struct Raw;
template <>
struct Raw<float> {
    float4 u, v;
    __device__ void zero() { u = v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ void load(const char* p, const char* q) {
        u = *reinterpret_cast<const float4*>(p);
        v = *reinterpret_cast<const float4*>(q);
    }
    __device__ static void store(char* p, char* q, const Raw& r) {
        *reinterpret_cast<float4*>(p) = r.u;
        *reinterpret_cast<float4*>(q) = r.v;
    }
    __device__ void load_one(int k, const char* p) {
        (&(k < 4 ? u : v).x)[k & 3] = *reinterpret_cast<const float*>(p);
    }
    __device__ void store_one(int k, char* p) const {
        *reinterpret_cast<float*>(p) = (&(k < 4 ? u : v).x)[k & 3];
    }
    template <int kPairs>
    __device__ Four get() const {
        if (kPairs == kNeighbours)
            return {{{u.x, u.z}, {v.x, v.z}}, {{u.y, u.w}, {v.y, v.w}}};
        return {{{u.x, u.y}, {u.z, u.w}}, {{v.x, v.y}, {v.z, v.w}}};
    }
    template <int kPairs>
    __device__ static Raw of(const Four& f) {
        Raw r;
        if (kPairs == kNeighbours) {
            r.u = make_float4(f.a[0].x, f.b[0].x, f.a[0].y, f.b[0].y);
            r.v = make_float4(f.a[1].x, f.b[1].x, f.a[1].y, f.b[1].y);
        } else {
            r.u = make_float4(f.a[0].x, f.a[0].y, f.a[1].x, f.a[1].y);
            r.v = make_float4(f.b[0].x, f.b[0].y, f.b[1].x, f.b[1].y);
        }
        return r;
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint2 u, v;
    __device__ void zero() { u = v = make_uint2(0, 0); }
    __device__ void load(const char* p, const char* q) {
        u = *reinterpret_cast<const uint2*>(p);
        v = *reinterpret_cast<const uint2*>(q);
    }
    __device__ static void store(char* p, char* q, const Raw& r) {
        *reinterpret_cast<uint2*>(p) = r.u;
        *reinterpret_cast<uint2*>(q) = r.v;
    }
    __device__ void load_one(int k, const char* p) {
        uint32_t& w = (k & 2) ? (k < 4 ? u.y : v.y) : (k < 4 ? u.x : v.x);
        const uint32_t h = *reinterpret_cast<const uint16_t*>(p);
        w = (k & 1) ? (w & 0xffffu) | (h << 16) : (w & 0xffff0000u) | h;
    }
    __device__ void store_one(int k, char* p) const {
        const uint32_t w = (k & 2) ? (k < 4 ? u.y : v.y) : (k < 4 ? u.x : v.x);
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)((k & 1) ? w >> 16 : w);
    }
    template <int kPairs>
    __device__ Four get() const {
        if (kPairs == kNeighbours)
            return {{{lo16(u.x), lo16(u.y)}, {lo16(v.x), lo16(v.y)}},
                    {{hi16(u.x), hi16(u.y)}, {hi16(v.x), hi16(v.y)}}};
        return {{{lo16(u.x), hi16(u.x)}, {lo16(u.y), hi16(u.y)}},
                {{lo16(v.x), hi16(v.x)}, {lo16(v.y), hi16(v.y)}}};
    }
    __device__ static uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    template <int kPairs>
    __device__ static Raw of(const Four& f) {
        Raw r;
        if (kPairs == kNeighbours) {
            r.u = make_uint2(pack(f.a[0].x, f.b[0].x), pack(f.a[0].y, f.b[0].y));
            r.v = make_uint2(pack(f.a[1].x, f.b[1].x), pack(f.a[1].y, f.b[1].y));
        } else {
            r.u = make_uint2(pack(f.a[0].x, f.a[0].y), pack(f.a[1].x, f.a[1].y));
            r.v = make_uint2(pack(f.b[0].x, f.b[0].y), pack(f.b[1].x, f.b[1].y));
        }
        return r;
    }
};

// Where a lane's four pairs lie in a row: pairs 4 l .. 4 l + 3, the rotated ones first.
template <int kPairs>
struct Cols {
    int first, second;  // columns of the two loads (kHalves4, kNeighbours)
    int pair;           // first pair
    int pairs;          // rotated pairs of a row
    int rot;

    __device__ __forceinline__ Cols(int lane, int rot_) : pair(4 * lane), pairs(rot_ >> 1), rot(rot_) {
        if (kPairs == kNeighbours) {
            first = 8 * lane;
            second = first + 4;
        } else {
            first = pair < pairs ? pair : rot + 2 * (pair - pairs);
            second = pair < pairs ? pair + pairs : first + 4;
        }
    }
    // column of value k of a lane's eight (the pairs' first values, then their second ones),
    // for any pairing: what kHalves reads one by one
    __device__ __forceinline__ int column(int k) const {
        const int g = pair + (k & 3);
        if (kPairs == kNeighbours) return 2 * g + (k >> 2);
        if (kPairs == kHalves4 && pair >= pairs) return k < 4 ? first + k : second + k - 4;
        return g < pairs ? g + (k < 4 ? 0 : pairs) : rot + 2 * (g - pairs) + (k >> 2);
    }
    template <typename T>
    __device__ __forceinline__ void load(Raw<T>& x, const char* row) const {
        if (kPairs != kHalves) {
            x.load(row + first * sizeof(T), row + second * sizeof(T));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x.load_one(k, row + column(k) * sizeof(T));
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(char* row, const Four& f) const {
        const Raw<T> r = Raw<T>::template of<kPairs>(f);
        if (kPairs != kHalves) {
            Raw<T>::store(row + first * sizeof(T), row + second * sizeof(T), r);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) r.store_one(k, row + column(k) * sizeof(T));
        }
    }
    // a lane's values of a row of fp32 (weights; 1 where there are none)
    __device__ __forceinline__ Four weights(const float* w) const {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = w ? __ldg(w + column(k)) : 1.f;
        return {{{v[0], v[1]}, {v[2], v[3]}}, {{v[4], v[5]}, {v[6], v[7]}}};
    }
    // cosines (a) and sines (b) of the four pairs (1 and 0 where not turned); a position beyond
    // the table shows in the result
    __device__ __forceinline__ Four angles(const HnParams& p, int64_t pos) const {
        float v[8] = {1.f, 1.f, 1.f, 1.f, 0.f, 0.f, 0.f, 0.f};
        if (pos >= 0 && pair < pairs) {
            const float* row = p.cos_sin + pos * rot;
            if (pos >= p.table_rows) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (pair + (k & 3) < pairs) v[k] = __int_as_float(0x7fc00000);
            } else if (pairs % 4 == 0) {  // whole 16-byte words
                const float4 c = __ldg(reinterpret_cast<const float4*>(row + pair));
                const float4 s = __ldg(reinterpret_cast<const float4*>(row + pairs + pair));
                v[0] = c.x, v[1] = c.y, v[2] = c.z, v[3] = c.w;
                v[4] = s.x, v[5] = s.y, v[6] = s.z, v[7] = s.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (pair + k < pairs) v[k] = __ldg(row + pair + k), v[4 + k] = __ldg(row + pairs + pair + k);
            }
        }
        return {{{v[0], v[1]}, {v[2], v[3]}}, {{v[4], v[5]}, {v[6], v[7]}}};
    }
};

__device__ __forceinline__ float2 neg(float2 v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// sum of a lane's eight products
__device__ __forceinline__ float inner(const Four& x, const Four& y) {
    float2 s = __fmul2_rn(x.a[0], y.a[0]);
    s = __ffma2_rn(x.a[1], y.a[1], s);
    s = __ffma2_rn(x.b[0], y.b[0], s);
    s = __ffma2_rn(x.b[1], y.b[1], s);
    return s.x + s.y;
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A warp's share: kRows rows a lane (of the queries' heads or the keys') of every step-th
// token.  Rows of fp32 take twice the registers.
template <typename T>
constexpr int kRows = sizeof(T) == 2 ? 2 : 1;

template <typename T, int kLanes>
struct Walker {
    static constexpr int kSub = 32 / kLanes, kHeads = kSub * kRows<T>;

    bool active, keys;
    int mine;   // rows of existing heads that the lane has
    int head0;  // the first; the others are kSub apart
    int64_t token;
    int step;

    __device__ __forceinline__ Walker(const HnParams& p) {
        const int sub = (threadIdx.x & 31) / kLanes;
        int w = blockIdx.x * kHnWarps + (threadIdx.x >> 5), part = 0;
        active = keys = false;
        token = 0;
        step = 1;
        // full parts of the queries, their last one, and the same of the keys
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const Share& s = p.share[k];
            if (!active && w < s.parts * s.warps) {
                active = true;
                keys = k >= 2;
                part = (k & 1 ? p.share[k - 1].parts : 0) + w / s.warps;
                token = w % s.warps;
                step = s.warps;
            }
            w -= s.parts * s.warps;
        }
        head0 = part * kHeads + sub;
        const int left = (keys ? p.hk : p.hq) - head0;
        mine = (int)(threadIdx.x & (kLanes - 1)) * 8 < p.dim ? min(kRows<T>, (left + kSub - 1) / kSub)
                                                            : 0;
    }
    __device__ __forceinline__ char* memory(const Rows& a) const {  // row of the first token
        return a.p + token * a.ts + head0 * a.hs;
    }
};

// a token's place in the table (a token later it is wanted: read ahead)
__device__ __forceinline__ int64_t position(const HnParams& p, int64_t t) {
    return t >= p.tokens ? (int64_t)-1 : p.positions ? (int64_t)__ldg(p.positions + t) : t;
}

template <typename T, int kPairs, int kLanes>
__global__ void __launch_bounds__(kHnThreads, 4) headnorm_kernel(const HnParams p) {
    grid_dep_sync();
    const Walker<T, kLanes> w(p);
    if (!w.active) return;
    const Rows in = w.keys ? p.k : p.q, out = w.keys ? p.yk : p.yq;
    const Cols<kPairs> c(threadIdx.x & (kLanes - 1), p.rot);
    const Four wt = c.weights(w.mine > 0 ? (w.keys ? p.kw : p.qw) : nullptr);
    const float inv_dim = 1.f / (float)p.dim;
    const char* src = w.memory(in);
    char* dst = w.memory(out);
    int64_t pos = position(p, w.token);
    for (int64_t t = w.token; t < p.tokens; t += w.step) {
        Raw<T> raw[kRows<T>];
#pragma unroll
        for (int r = 0; r < kRows<T>; ++r) {
            raw[r].zero();
            if (r < w.mine) c.load(raw[r], src + r * (w.kSub * in.hs));
        }
        const Four turn = c.angles(p, pos);
        pos = position(p, t + w.step);
        float2 aa[2], ab[2], bb[2], ba[2];  // factors: a from a, a from b, b from b, b from a
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            aa[k] = __fmul2_rn(turn.a[k], wt.a[k]);
            ab[k] = neg(__fmul2_rn(turn.b[k], wt.b[k]));
            bb[k] = __fmul2_rn(turn.a[k], wt.b[k]);
            ba[k] = __fmul2_rn(turn.b[k], wt.a[k]);
        }
        __syncwarp();  // rows may be overwritten in place: all of them are read
#pragma unroll
        for (int r = 0; r < kRows<T>; ++r) {
            const Four x = raw[r].template get<kPairs>();
            const float s = row_sum<kLanes>(inner(x, x));
            const float2 rn = both(rsqrtf(fmaf(s, inv_dim, p.eps)));
            Four o;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                o.a[k] = __fmul2_rn(rn, __ffma2_rn(x.b[k], ab[k], __fmul2_rn(x.a[k], aa[k])));
                o.b[k] = __fmul2_rn(rn, __ffma2_rn(x.a[k], ba[k], __fmul2_rn(x.b[k], bb[k])));
            }
            if (r < w.mine) c.template store<T>(dst + r * (w.kSub * out.hs), o);
        }
        src += w.step * in.ts;
        dst += w.step * out.ts;
    }
}

template <typename T, int kPairs, int kLanes>
__global__ void __launch_bounds__(kHnThreads, 3) headnorm_bwd_kernel(const HnParams p) {
    grid_dep_sync();
    __shared__ float sum[kHnWarps][kLanes * 8];
    __shared__ int side_of[kHnWarps];
    const Walker<T, kLanes> w(p);
    const Cols<kPairs> c(threadIdx.x & (kLanes - 1), p.rot);
    Four dw{};
    if (w.active) {
        const Rows in = w.keys ? p.k : p.q, gy = w.keys ? p.yk : p.yq, out = w.keys ? p.dk : p.dq;
        const Four wt = c.weights(w.mine > 0 ? (w.keys ? p.kw : p.qw) : nullptr);
        const float inv_dim = 1.f / (float)p.dim;
        const char *src = w.memory(in), *src_d = w.memory(gy);
        char* dst = w.memory(out);
        int64_t pos = position(p, w.token);
        for (int64_t t = w.token; t < p.tokens; t += w.step) {
            Raw<T> raw[kRows<T>], raw_d[kRows<T>];
#pragma unroll
            for (int r = 0; r < kRows<T>; ++r) {
                raw[r].zero();
                raw_d[r].zero();
                if (r < w.mine) {
                    c.load(raw[r], src + r * (w.kSub * in.hs));
                    c.load(raw_d[r], src_d + r * (w.kSub * gy.hs));
                }
            }
            const Four turn = c.angles(p, pos);
            pos = position(p, t + w.step);
            __syncwarp();  // the gradient may come over dy or x: all of the rows is read
#pragma unroll
            for (int r = 0; r < kRows<T>; ++r) {
                const Four x = raw[r].template get<kPairs>(), d = raw_d[r].template get<kPairs>();
                Four g, wg;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    g.a[k] = __ffma2_rn(d.b[k], turn.b[k], __fmul2_rn(d.a[k], turn.a[k]));
                    g.b[k] = __ffma2_rn(neg(d.a[k]), turn.b[k], __fmul2_rn(d.b[k], turn.a[k]));
                    wg.a[k] = __fmul2_rn(g.a[k], wt.a[k]);
                    wg.b[k] = __fmul2_rn(g.b[k], wt.b[k]);
                }
                const float s = row_sum<kLanes>(inner(x, x));
                const float dot = row_sum<kLanes>(inner(x, wg));
                const float rn = rsqrtf(fmaf(s, inv_dim, p.eps));
                const float2 r2 = both(rn), m2 = both(-dot * inv_dim * rn * rn);
                if (r < w.mine) {
                    Four o;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        o.a[k] = __fmul2_rn(r2, __ffma2_rn(x.a[k], m2, wg.a[k]));
                        o.b[k] = __fmul2_rn(r2, __ffma2_rn(x.b[k], m2, wg.b[k]));
                        dw.a[k] = __ffma2_rn(g.a[k], __fmul2_rn(x.a[k], r2), dw.a[k]);
                        dw.b[k] = __ffma2_rn(g.b[k], __fmul2_rn(x.b[k], r2), dw.b[k]);
                    }
                    c.template store<T>(dst + r * (w.kSub * out.hs), o);
                }
            }
            src += w.step * in.ts;
            src_d += w.step * gy.ts;
            dst += w.step * out.ts;
        }
    }
    // the warp's rows, then the block's warps of the same side, in order
    const int warp = threadIdx.x >> 5;
    const float v[8] = {dw.a[0].x, dw.a[0].y, dw.a[1].x, dw.a[1].y,
                        dw.b[0].x, dw.b[0].y, dw.b[1].x, dw.b[1].y};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float a = v[k];
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if ((threadIdx.x & 31) < kLanes && c.pair * 2 < p.dim) sum[warp][c.column(k)] = a;
    }
    if ((threadIdx.x & 31) == 0) side_of[warp] = !w.active ? -1 : w.keys;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.dim; i += kHnThreads) {
        const int side = i >= p.dim, e = side ? i - p.dim : i;
        float s = 0.f;
        for (int u = 0; u < kHnWarps; ++u)
            if (side_of[u] == side) s += sum[u][e];
        p.part[(int64_t)blockIdx.x * 2 * p.dim + i] = s;
    }
}

// dw[side][e] = the blocks' sums: 32 threads take every 32nd block of a column, and their
// sums are added in order
__global__ void __launch_bounds__(kFinishThreads)
    headnorm_finish_kernel(const float* __restrict__ part, int blocks, int dim, float* dqw,
                           float* dkw) {
    grid_dep_sync();
    constexpr int kOf = kFinishThreads / kFinishCols;
    __shared__ float s[kOf][kFinishCols];
    const int col = threadIdx.x % kFinishCols, row = threadIdx.x / kFinishCols;
    const int i = blockIdx.x * kFinishCols + col;
    float a = 0.f;
    if (i < 2 * dim) {
#pragma unroll
        for (int k = 0; k < (kBwdBlocks + kOf - 1) / kOf; ++k) {
            const int b = row + k * kOf;
            if (b < blocks) a += __ldg(part + (int64_t)b * 2 * dim + i);
        }
    }
    s[row][col] = a;
    __syncthreads();
    if (row == 0 && i < 2 * dim) {
        for (int r = 1; r < kOf; ++r) a += s[r][col];
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

template <typename T, int kPairs, int kLanes, bool kBwd>
cudaError_t launch_lanes(HnParams p, int* blocks_out, cudaStream_t st) {
    using W = Walker<T, kLanes>;
    // warps by the rows that a part's lanes have, or one a token where there are enough
    constexpr int64_t kMostWarps = (int64_t)(kBwd ? kBwdBlocks : kFwdBlocks) * kHnWarps;
    int rows[4];
    int64_t parts = 0, all_rows = 0, warps = 0;
    for (int side = 0; side < 2; ++side) {
        const int heads = side ? p.hk : p.hq, full = (heads - 1) / W::kHeads;
        p.share[2 * side].parts = full;
        p.share[2 * side + 1].parts = 1;
        rows[2 * side] = kRows<T>;
        rows[2 * side + 1] = (heads - full * W::kHeads + W::kSub - 1) / W::kSub;
    }
    for (int k = 0; k < 4; ++k) {
        parts += p.share[k].parts;
        all_rows += p.share[k].parts * rows[k];
    }
    for (int k = 0; k < 4; ++k) {
        Share& s = p.share[k];
        const int64_t fair = std::max<int64_t>(1, kMostWarps * rows[k] / all_rows);
        s.warps = (int)(p.tokens * parts <= kMostWarps ? std::max<int64_t>(1, p.tokens)
                                                       : std::min(fair, p.tokens));
        warps += (int64_t)s.parts * s.warps;
    }
    const int blocks = (int)((warps + kHnWarps - 1) / kHnWarps);
    *blocks_out = blocks;
    void (*kernel)(const HnParams) =
        kBwd ? headnorm_bwd_kernel<T, kPairs, kLanes> : headnorm_kernel<T, kPairs, kLanes>;
    return launch(kernel, dim3(blocks), dim3(kHnThreads), 0, st, p);
}

template <typename T, int kPairs, bool kBwd>
cudaError_t launch_pairs(const HnParams& p, int* blocks, cudaStream_t st) {
    switch (lanes_of(p.dim)) {
        case 1: return launch_lanes<T, kPairs, 1, kBwd>(p, blocks, st);
        case 2: return launch_lanes<T, kPairs, 2, kBwd>(p, blocks, st);
        case 4: return launch_lanes<T, kPairs, 4, kBwd>(p, blocks, st);
        case 8: return launch_lanes<T, kPairs, 8, kBwd>(p, blocks, st);
        case 16: return launch_lanes<T, kPairs, 16, kBwd>(p, blocks, st);
        default: return launch_lanes<T, kPairs, 32, kBwd>(p, blocks, st);
    }
}

template <typename T, bool kBwd>
cudaError_t launch_typed(const HeadNormArgs& a, const HnParams& p, int* blocks, cudaStream_t st) {
    if (a.interleaved) return launch_pairs<T, kNeighbours, kBwd>(p, blocks, st);
    return a.rot % 8 == 0 ? launch_pairs<T, kHalves4, kBwd>(p, blocks, st)
                           : launch_pairs<T, kHalves, kBwd>(p, blocks, st);
}

template <bool kBwd>
cudaError_t launch_any(const HeadNormArgs& a, const HnParams& p, int* blocks, cudaStream_t st) {
    return a.bf16 ? launch_typed<__nv_bfloat16, kBwd>(a, p, blocks, st)
                  : launch_typed<float, kBwd>(a, p, blocks, st);
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
    return (size_t)kBwdBlocks * 2 * dim * sizeof(float);
}

cudaError_t launch_headnorm(const HeadNormArgs& a, const gs_heads& q, const gs_heads& k,
                            const gs_heads& q_out, const gs_heads& k_out, cudaStream_t st) {
    int blocks = 0;
    return launch_any<false>(a, params_of(a, q, k, q_out, k_out), &blocks, st);
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
    const cudaError_t e = launch_any<true>(a, p, &blocks, st);
    if (e != cudaSuccess || (!dqw && !dkw)) return e;
    return launch(headnorm_finish_kernel, dim3((2 * a.dim + kFinishCols - 1) / kFinishCols),
                  dim3(kFinishThreads), 0, st, static_cast<const float*>(p.part), blocks, a.dim, dqw,
                  dkw);
}

}  // namespace gs
