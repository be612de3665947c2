// gs_attention_tokens.cu -- attention over a window of keys and sinks for few queries: one token or
// some of every sequence, as where tokens are predicted one after the other.
//
//   out = sum_j softmax_j(scale q . k_j) v_j  over the keys that the query sees
//
// Memory bounds it: every key and value that is seen is read once, for all query heads that share it.
// A block takes a query and a key head (up to 8 of the heads that share it), a cluster of blocks and
// the warps in them divide the keys, 16 at a step.  The products go over the tensor cores with the
// heads as the narrow side of 8,
//   S^T [16 keys x 8] = K Q^T,  O^T [16 values x 8] += V^T P^T,
// so that keys and values go from memory straight into operand registers, in 16-byte words: a lane
// holds the same words of a key's and of a query's row, and the contraction runs over them in
// whatever order they lie.  V^T and P^T are 8 x 8 blocks turned around between registers.  Warps keep
// their own running maximum and sum; the blocks join them in shared memory, the cluster its blocks'
// over distributed shared memory: one launch, no workspace.
//
// Measured: 32 tokens, 16 heads on 4 x 128, 2,048 keys and 4 sinks each, 130 MB: 31.3 us, 4.2 TB/s;
// 64 tokens 53 us, 5.0 TB/s, with 8 warps' loads of 16 keys ahead on two blocks an SM.  What is left is
// the start (the sequence's place, then the first keys: two latencies) and the join of the blocks.
//
// As in gs_attention_fwd.cu the maximum may lag by 8 in powers of two, P is rounded to bfloat16 for
// its product, everything else is fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gs_attention.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {
namespace {

constexpr int kTokenWarps = 8;
constexpr int kTokenThreads = kTokenWarps * 32;
constexpr int kRows = 8;    // query heads of a block
constexpr int kStep = 16;   // keys a warp takes at once
constexpr int kMostSplits = 8;  // blocks of a cluster
constexpr int kSms = 152;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kStale = 8.f;  // powers of two by which a maximum may rise unnoticed

struct TokenParams {
    Batch batch;
    Window window;
    int heads_k, group, parts;  // parts: of 8 heads that share a key head
    int dim, splits;
    float log2_scale;  // scale log2(e)
    HeadView q, k, v, o;
    float* lse;
};

// D += A B, A [16 x 16] rows, B [16 x 8] columns, bfloat16, D fp32
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// an 8 x 8 block of 16-bit values, a row to four lanes, turned around
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float of the same place in the shared memory of the cluster's block `rank`
__device__ __forceinline__ float of_block(const float* at, int rank) {
    uint32_t addr;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// By one whole warp: the sequence that holds query token t (-1: none), in as many rounds as the
// batch has powers of 32.
__device__ __forceinline__ int sequence_of(const Batch& v, int64_t t, Sequence* sq) {
    if (!v.cu_q) {
        *sq = sequence(v, 0);
        return 0;
    }
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = v.batch;  // the last sequence that starts at the token or before
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, b = lo + lane * step;
        const unsigned upto = __ballot_sync(0xffffffffu, b < hi && __ldg(v.cu_q + b) <= t);
        if (upto) lo += (31 - __clz(upto)) * step;
        hi = min(hi, lo + step);
    }
    *sq = sequence(v, lo);
    return t >= sq->q0 && t < sq->q0 + sq->n ? lo : -1;
}

// A lane's words of a row: 16-byte word (lane % 4) + 4 i, zeros beyond the row.
template <int kWords>
struct Words {
    uint4 w[kWords];
    __device__ __forceinline__ void load(const __nv_bfloat16* row, int dim) {
        const int c = threadIdx.x & 3;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (row && (c + 4 * i) * 8 < dim)
                w[i] = __ldg(reinterpret_cast<const uint4*>(row) + c + 4 * i);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ uint32_t at(int i, int j) const {
        return j == 0 ? w[i].x : j == 1 ? w[i].y : j == 2 ? w[i].z : w[i].w;
    }
};

// kWords: 16-byte words a lane of a row, for rows of up to 32 kWords values.
template <int kWords>
__global__ void __launch_bounds__(kTokenThreads, 2) attention_tokens_kernel(const TokenParams p) {
    grid_dep_sync();
    constexpr int kDim = 32 * kWords;
    __shared__ float tops[kTokenWarps][kRows], sums[kTokenWarps][kRows];
    __shared__ float outs[kTokenWarps][kRows][kDim];  // the first warp's place: the block's
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3, r = lane >> 2;
    const int split = (int)(blockIdx.x % p.splits);
    const int64_t item = blockIdx.x / p.splits;
    const int part = (int)(item % p.parts), khead = (int)(item / p.parts % p.heads_k);
    const int64_t token = item / p.parts / p.heads_k;
    const int head0 = khead * p.group + part * kRows, heads = min(kRows, p.group - part * kRows);
    Sequence sq;
    const bool held = sequence_of(p.batch, token, &sq) >= 0;
    Seen see{0, 0, 0};
    if (held) see = seen_by(p.window, (int)(token - sq.q0), sq.n, sq.m);
    // the keys seen in their order: the sinks, then the window; as one where they meet
    if (see.sinks >= see.lo) {
        see.hi = max(see.hi, see.sinks);
        see.lo = see.sinks = 0;
    }
    const int before = see.sinks;
    const int keys = before + see.hi - see.lo;
    const auto key_of = [&](int i) {
        i = min(i, keys - 1);  // beyond the last one it again, with probability 0
        return i < before ? i : see.lo + i - before;
    };

    Words<kWords> q;
    q.load(r < heads ? p.q.row(token, head0 + r) : nullptr, p.dim);
    float o[kWords][2][4] = {};
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};  // of rows 2 c and 2 c + 1
    Words<kWords> k0, k1, v0, v1;  // of keys r and r + 8 of the step
    const int stride = p.splits * kTokenWarps * kStep;
    int at = (split * kTokenWarps + warp) * kStep;
    const auto load = [&](Words<kWords>& a, Words<kWords>& b, const HeadView& of, int i) {
        a.load(of.row(sq.k0 + key_of(i + r), khead), p.dim);
        b.load(of.row(sq.k0 + key_of(i + r + 8), khead), p.dim);
    };
    if (at < keys) {
        load(k0, k1, p.k, at);
        load(v0, v1, p.v, at);
    }
    for (; at < keys; at += stride) {
        float s[4] = {};
#pragma unroll
        for (int i = 0; i < kWords; ++i)
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                mma16816(s, k0.at(i, j), k1.at(i, j), k0.at(i, j + 1), k1.at(i, j + 1), q.at(i, j),
                         q.at(i, j + 1));
        if (at + stride < keys) load(k0, k1, p.k, at + stride);
        // s: keys r, r, r + 8, r + 8 with rows 2 c, 2 c + 1 in turn
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[e] *= p.log2_scale;
            if (at + r + (e >> 1) * 8 >= keys) s[e] = -INFINITY;
        }
        float high[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
        for (int e = 4; e < 32; e <<= 1) {
            high[0] = fmaxf(high[0], __shfl_xor_sync(0xffffffffu, high[0], e));
            high[1] = fmaxf(high[1], __shfl_xor_sync(0xffffffffu, high[1], e));
        }
        const bool risen = high[0] - top[0] > kStale || high[1] - top[1] > kStale;
        if (__any_sync(0xffffffffu, risen)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = high[e] > top[e] ? ex2_approx(top[e] - high[e]) : 1.f;
                top[e] = fmaxf(top[e], high[e]);
                sum[e] *= f;
#pragma unroll
                for (int i = 0; i < kWords; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        o[i][j][e] *= f;
                        o[i][j][e + 2] *= f;
                    }
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (by the score, not by the maximum: a row of NaN has none)
            s[e] = s[e] == -INFINITY ? 0.f : ex2_approx(s[e] - top[e & 1]);
            sum[e & 1] += s[e];
        }
        // values behind the last key are the last one's, with probability 0: zeros instead, which that
        // leaves out whatever they are.  (Loaded as zeros: up to 7 % more for every step's choice.)
        if (at + kStep > keys) {
            if (at + r >= keys) v0.clear();
            if (at + r + 8 >= keys) v1.clear();
        }
        const uint32_t p0 = transposed(pack_bf16(s[0], s[1])), p1 = transposed(pack_bf16(s[2], s[3]));
#pragma unroll
        for (int i = 0; i < kWords; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                mma16816(o[i][j], transposed(v0.at(i, 2 * j)), transposed(v0.at(i, 2 * j + 1)),
                         transposed(v1.at(i, 2 * j)), transposed(v1.at(i, 2 * j + 1)), p0, p1);
        if (at + stride < keys) load(v0, v1, p.v, at + stride);
    }
    // ---- the warps' results, each in its place ----
#pragma unroll
    for (int e = 4; e < 32; e <<= 1) {
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], e);
        sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], e);
    }
    if (r == 0)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            tops[warp][2 * c + e] = top[e];
            sums[warp][2 * c + e] = sum[e];
        }
    // block (i, j) holds values 32 i + 8 (r / 2) + r % 2 + 4 j (+ 2) of rows 2 c and 2 c + 1
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                outs[warp][2 * c + (e & 1)][32 * i + 8 * (r >> 1) + (r & 1) + 4 * j + (e & 2)] =
                    o[i][j][e];
    __syncthreads();
    // ---- the block's, in the first warp's place: a warp a row ----
    {
        float most = tops[0][warp];
#pragma unroll
        for (int w = 1; w < kTokenWarps; ++w) most = fmaxf(most, tops[w][warp]);
        float f[kTokenWarps], l = 0.f;
#pragma unroll
        for (int w = 0; w < kTokenWarps; ++w) {
            f[w] = tops[w][warp] == -INFINITY ? 0.f : ex2_approx(tops[w][warp] - most);
            l = fmaf(f[w], sums[w][warp], l);
        }
        for (int d = lane; d < kDim; d += 32) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kTokenWarps; ++w) a = fmaf(f[w], outs[w][warp][d], a);
            outs[0][warp][d] = a;
        }
        __syncwarp();
        if (lane == 0) tops[0][warp] = most, sums[0][warp] = l;
    }
    // ---- the cluster's: its blocks take the rows in turn ----
    if (p.splits > 1)
        cluster_sync();
    else
        __syncthreads();
    for (int row = split + warp * p.splits; row < heads && held; row += kTokenWarps * p.splits) {
        float most = -INFINITY, l = 0.f, f[kMostSplits];
        float top_of[kMostSplits];
#pragma unroll
        for (int b = 0; b < kMostSplits; ++b) {
            top_of[b] = -INFINITY;
            if (b < p.splits) top_of[b] = p.splits > 1 ? of_block(&tops[0][row], b) : tops[0][row];
            most = fmaxf(most, top_of[b]);
        }
#pragma unroll
        for (int b = 0; b < kMostSplits; ++b) {
            f[b] = top_of[b] == -INFINITY ? 0.f : ex2_approx(top_of[b] - most);
            if (b < p.splits)
                l = fmaf(f[b], p.splits > 1 ? of_block(&sums[0][row], b) : sums[0][row], l);
        }
        const float scale = l != 0.f ? 1.f / l : 0.f;
        __nv_bfloat16* out = p.o.row(token, head0 + row);
        for (int d = 2 * lane; d < p.dim; d += 64) {
            float a = 0.f, b2 = 0.f;
#pragma unroll
            for (int b = 0; b < kMostSplits; ++b)
                if (b < p.splits) {
                    const float* from = &outs[0][row][d];
                    a = fmaf(f[b], p.splits > 1 ? of_block(from, b) : from[0], a);
                    b2 = fmaf(f[b], p.splits > 1 ? of_block(from + 1, b) : from[1], b2);
                }
            *reinterpret_cast<uint32_t*>(out + d) = pack_bf16(a * scale, b2 * scale);
        }
        if (lane == 0)
            p.lse[(int64_t)(head0 + row) * p.batch.tq + token] =
                l != 0.f ? (most + log2f(l)) * kLn2 : -INFINITY;
    }
    if (p.splits > 1) cluster_sync();  // no block's memory goes while another reads it
}

template <int kWords>
cudaError_t launch_words(const TokenParams& p, int64_t items, cudaStream_t st) {
    return launch_clustered(attention_tokens_kernel<kWords>, (unsigned)p.splits,
                            dim3((unsigned)(items * p.splits)), dim3(kTokenThreads), 0, st, p);
}

}  // namespace

// Few queries a sequence, on average.  A query's keys are read for it alone but for all heads that
// share them; tiles of 128 queries cost the same for one as for many, but each head its own.  So the
// queries from which on tiles go faster rise with the heads on a key head.  (8,000 to 32,400 keys, 1,024
// to 8,192 of them seen, 16 heads on 4 x 128, 1, 2, 4, 8 queries of each of 32 sequences: 31, 43, 75,
// 139 us here, 118 to 126 by tiles; 8 x 64 on as many, 513 keys, 128 sequences, 1, 2, 3: 37, 58, 83 and
// 64 by tiles.)
// The host knows no lengths, so a batch of mixed ones goes by its average.  Single queries beside a prompt
// are still better off here while windows are short, and up to three times worse where most queries are
// one sequence's: 31 tokens on 8,000 keys and 129 queries on 32,400, as many heads, 1,024, 2,048, 32,400 of
// the keys seen: 52, 90, 990 us here, 77, 129, 695 by tiles; 160 queries on 32,400 keys among 31 empty
// sequences: 50, 88, 1,275 and 25, 38, 400.
bool few_queries(const gs_attention_shape& s) {
    const int64_t few = 1 + std::min(s.heads_q / s.heads_k, 4);
    return s.tokens_q <= few * s.batch && s.tokens_q * s.heads_q <= (int64_t(1) << 27);
}

cudaError_t launch_attention_tokens(const gs_attention_shape& s, const gs_window& window,
                                    const gs_heads& q, const gs_heads& k, const gs_heads& v,
                                    const gs_heads& out, float* lse, const int32_t* cu_q,
                                    const int32_t* cu_k, cudaStream_t st) {
    const auto view = [](const gs_heads& h) {
        return HeadView{static_cast<__nv_bfloat16*>(h.data), h.token_stride, h.head_stride};
    };
    TokenParams p{};
    p.batch = {cu_q, cu_k, s.tokens_q, s.tokens_k, s.batch, false};
    p.window = window_of(window, s.causal != 0);
    p.heads_k = s.heads_k;
    p.group = s.heads_q / s.heads_k;
    p.parts = (p.group + kRows - 1) / kRows;
    p.dim = s.head_dim;
    p.log2_scale = s.scale * 1.4426950408889634f;
    p.q = view(q);
    p.k = view(k);
    p.v = view(v);
    p.o = view(out);
    p.lse = lse;
    const int64_t items = s.tokens_q * s.heads_k * p.parts;
    // as many blocks as run at once, two an SM, as long as every warp has keys
    const int64_t keys =
        std::min<int64_t>(s.tokens_k, (int64_t)window.left + window.right + 1 + window.sinks);
    p.splits = (int)std::max<int64_t>(
        1, std::min<int64_t>({kMostSplits, 2 * kSms / std::max<int64_t>(items, 1),
                              (keys + kTokenWarps * kStep - 1) / (kTokenWarps * kStep)}));
    switch ((s.head_dim + 31) / 32) {
        case 1: return launch_words<1>(p, items, st);
        case 2: return launch_words<2>(p, items, st);
        case 3: return launch_words<3>(p, items, st);
        default: return launch_words<4>(p, items, st);
    }
}

}  // namespace gs
