// gs_attention_bwd.cu -- the gradient of softmax attention on the tensor cores, with the
// probabilities recomputed from the forward's row sums.
//
//   P = exp(scale Q K^T - lse),  dV = P^T dO,  dS = P (dO V^T - delta),
//   dQ = scale dS K,  dK = scale dS^T Q,  delta_i = O_i . dO_i
//
// Two kernels.  The first makes delta.  The second has blocks of two kinds.  One takes 128
// keys and walks the queries of every head that shares them: dK and dV stay in tensor memory,
// so the sum over a group's heads and over queries needs no atomics.  The other takes 128
// queries and walks the keys, with dQ in tensor memory.  S and dO V^T are formed in both:
// seven products instead of five.  The other way, dQ added to memory from the blocks of keys,
// moves 64 KB of fp32 additions per 128 x 128 tile, about as many bytes per clock as L2
// takes, and its result would depend on their order.  Neither kind needs anything of the
// other, and in one launch the blocks of queries fill the last wave of the blocks of keys.
//
// What bounds them, at 128 values a head: a step of a block of keys is 2,048 cycles of
// products and as many of shared memory at 128 bytes a cycle (192 KB of operands, 64 KB that
// TMA writes), a step of a block of queries 1,536; the tensor pipe is busy 72 % of the active
// time, and leaving out all arithmetic between the products saves 7 %.  8,160 tokens x 16 heads
// on 4, called one by one: 1,127 us with the row sums, 1,210 TFLOP/s of the gradient's
// five products, 1,694 of the seven that are done (0.91 of the rate that the library's matrix
// product reaches in single calls); back to back, under the power limit: 1,183 to 1,205 us from
// card to card (0.92 to 0.94 of the library's rate under it).  At 64 values: 846 us one by one;
// there the handshakes bound it.
//
// The transposes come out of the operand descriptors: a tile of rows in shared memory
// serves both as an operand contracted along its columns and as one contracted along its
// rows.  P^T and dS^T (blocks of keys) and dS (of queries) go back to tensor memory in bfloat16
// over the scores they came from, as first operands.  P, dP - delta and the sums are fp32; P
// and dS are rounded to bfloat16 once, for the products, whose other operands are the caller's
// bfloat16 dO, Q and K.  By norms the gradients stand 0.0023 to 0.0025 from the exact ones, where
// rounding the exact ones to bfloat16 alone gives 0.0016 to 0.0018; exact arithmetic with P and
// dS rounded gives the same as the kernel.
//
// Rows of a tile that lie beyond the sequence and are contracted over are zeroed in shared
// memory, and P and dS are set to zero there by selection, so that what lies behind a
// sequence (NaN included) does not reach it.
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

constexpr int kMathWarps = 8;
constexpr int kBwdThreads = (kMathWarps + 2) * 32;
constexpr int kDeltaThreads = 256;

// Blocks `whole` .. `whole` + `rest` - 1 are cut into `pieces` of `chunk` tiles of the other
// side, a block each, piece by piece; a kernel adds the pieces' fp32 results up.
constexpr int kSms = 152;
struct BwdPlan {
    int64_t whole, rest;
    int chunk, pieces;
    int slot_rows;  // rows that a piece keeps in the workspace
};

// What a block works on, kept in shared memory: registers are short in the inner loops.
struct BwdWork {
    Sequence sq;
    int row0;         // first key (dK, dV) or query (dQ) of the block in its sequence
    int head, khead;
    int first, items; // tiles of the other side: those of the block's piece
    int64_t part;     // first row in the workspace (-1: the block writes the output itself)
};

struct BwdParams {
    Batch batch;
    int heads_q, heads_k, group, dim;
    bool negative, swap_q, swap_k, swap_v, swap_d;
    float scale, log2_scale;  // scale, and |scale| log2(e)
    HeadView o, dout, dq, dk, dv;
    const float* lse;
    float *nlse, *ndelta;  // [heads][tokens]: -lse log2(e) (-infinity: saw no key), -delta
    unsigned int* gave_up;
    BwdPlan plan_k, plan_q;     // of the blocks of keys, of queries
    float *parts_k, *parts_q;   // [pieces][rest][slot_rows][DP]: dK, then dV; dQ
};

// query tiles that see a block of keys, for each head of the group: from *first on
__device__ __forceinline__ int queries_of(const Sequence& sq, int key0, bool causal, int* first) {
    const int tiles = (sq.n + kTileRows - 1) / kTileRows;
    *first = causal ? min(tiles, max(0, key0 + sq.n - sq.m) / kTileRows) : 0;
    return tiles - *first;
}

// key tiles that a block of queries sees
__device__ __forceinline__ int keys_of(const Sequence& sq, int row0, bool causal) {
    const int last = min(sq.n, row0 + kTileRows) - 1;
    return (seen_keys(last, sq.n, sq.m, causal) + kTileRows - 1) / kTileRows;
}

__host__ __device__ inline int64_t part_rows(const BwdPlan& plan) {
    return plan.pieces > 1 ? plan.pieces * plan.rest * plan.slot_rows : 0;
}

__host__ __device__ inline int64_t blocks_of(const BwdPlan& plan) {
    return plan.whole + plan.rest * plan.pieces;
}

// By one whole warp: the work of block `id` of its kind, or false.
template <bool kKeys>
__device__ __forceinline__ bool find_work(const BwdParams& p, int64_t id, BwdWork* out) {
    const BwdPlan& plan = kKeys ? p.plan_k : p.plan_q;
    int64_t part = -1;
    int piece = 0;
    if (id >= plan.whole) {  // the cut blocks, piece by piece
        part = (id - plan.whole) * plan.slot_rows;
        piece = (int)((id - plan.whole) / plan.rest);
        id -= piece * plan.rest;
    }
    Place at{};
    if (!find_place<kKeys>(p.batch, kTileRows, kKeys ? p.heads_k : p.heads_q, (int)id, &at))
        return false;
    BwdWork w;
    w.sq = at.sq;
    w.row0 = at.tile * kTileRows;
    w.head = at.head;
    w.khead = kKeys ? at.head : at.head / p.group;
    int unused;
    w.items = kKeys ? queries_of(w.sq, w.row0, p.batch.causal, &unused) * p.group
                    : keys_of(w.sq, w.row0, p.batch.causal);
    w.first = 0;
    w.part = part;
    if (part >= 0) {
        w.first = piece * plan.chunk;
        w.items = min(max(w.items - w.first, 0), plan.chunk);
        if (piece > 0 && w.items == 0) return false;
    }
    if ((threadIdx.x & 31) == 0) *out = w;
    return true;
}


// ---------------------------------------------------------------------------
// -lse log2(e) and -delta of every query row
// ---------------------------------------------------------------------------
// 16 lanes a row; -infinity for a row that saw no key, so that its P comes out 0
__global__ void __launch_bounds__(kDeltaThreads) attention_delta_kernel(const BwdParams p) {
    grid_dep_sync();
    const int64_t at = ((int64_t)blockIdx.x * kDeltaThreads + threadIdx.x) >> 4;
    const int lane = threadIdx.x & 15;
    const int64_t t = at / p.heads_q;
    const int h = (int)(at - t * p.heads_q);
    float s = 0.f;
    if (t < p.batch.tq && lane * 8 < p.dim) {
        const uint4 a = *reinterpret_cast<const uint4*>(p.o.row(t, h) + lane * 8);
        const uint4 b = *reinterpret_cast<const uint4*>(p.dout.row(t, h) + lane * 8);
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s = fmaf(__uint_as_float(x[k] << 16), __uint_as_float(y[k] << 16), s);
            s = fmaf(__uint_as_float(x[k] & 0xffff0000u), __uint_as_float(y[k] & 0xffff0000u), s);
        }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (t < p.batch.tq && lane == 0) {
        const float l = p.lse[h * p.batch.tq + t];
        p.nlse[h * p.batch.tq + t] = l == -INFINITY ? l : l * -1.4426950408889634f;
        p.ndelta[h * p.batch.tq + t] = -s;
    }
}

// 64 values of a row of tensor memory, in bfloat16, over the first 32 of the 64 columns
__device__ __forceinline__ void store_half(uint32_t at, const float* v) {
    uint32_t w[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
    tmem_st32(at, w);
}

// kDim columns of a row of tensor memory (or zeros), times f, to memory: in bfloat16 to `out`,
// or as they are to `part`
template <int kDim>
__device__ __forceinline__ void store_row(uint32_t at, __nv_bfloat16* out, float* part, int dim,
                                          float f, bool zero) {
#pragma unroll
    for (int c = 0; c < kDim; c += 32) {
        uint32_t o[32];
        if (!zero) {
            tmem_ld32(o, at + c);
            tmem_wait_ld();
        }
        if (part) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
                *reinterpret_cast<uint4*>(part + c + k) =
                    zero ? make_uint4(0, 0, 0, 0) : make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
        if (!out) continue;
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
            if (c + k < dim) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = zero ? 0u
                                : pack_bf16(__uint_as_float(o[k + 2 * e]) * f,
                                            __uint_as_float(o[k + 2 * e + 1]) * f);
                *reinterpret_cast<uint4*>(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// dK and dV
// ---------------------------------------------------------------------------
template <int DP>
struct DkvShape {
    static constexpr int kBlocks = DP / kBlockCols;
    static constexpr uint32_t kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kSlots = DP == 128 ? 2 : 4;
    // dO V^T tiles in tensor memory, beside S, dV and dK: with two the next one is formed
    // before dS of this one is
    static constexpr int kDp = DP == 128 ? 1 : 2;
    static constexpr uint32_t kRows = (2 + 2 * kSlots) * kTileBytes;  // behind the tiles
    static constexpr uint32_t kSmem = kRows + kSlots * 2 * kTileRows * sizeof(float) + 1024;
};

template <int DP>
__device__ __forceinline__ void dkv_block(const CUtensorMap& map_q, const CUtensorMap& map_k,
                                          const CUtensorMap& map_v, const CUtensorMap& map_d,
                                          const BwdParams& p, int64_t id) {
    using Sh = DkvShape<DP>;
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bar_k, bar_v, bar_s, bar_dp[Sh::kDp], bar_p, bar_ds[Sh::kDp], bar_done,
        bar_raw, bar_drain;
    __shared__ uint64_t full_q[Sh::kSlots], empty_q[Sh::kSlots], full_d[Sh::kSlots],
        empty_d[Sh::kSlots];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    __shared__ BwdWork work;
    __shared__ int found;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const bool ok = find_work<true>(p, id, &work);
        if (lane == 0) found = ok, dead = 0;
    }
    __syncthreads();
    if (!found) return;
    const int items = work.items;

    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t at_k = smem, at_v = smem + Sh::kTileBytes;
    const uint32_t at_q = smem + 2 * Sh::kTileBytes, at_d = at_q + Sh::kSlots * Sh::kTileBytes;
    // -lse log2(e) and -delta of each slot's queries
    auto* rows = reinterpret_cast<float(*)[2][kTileRows]>(
        smem_raw + (smem + Sh::kRows - smem_u32(smem_raw)));
    if (warp == kMathWarps) {
        tmem_alloc(smem_u32(&tmem_at), 512);
    } else if (threadIdx.x == 0) {
        for (uint64_t* b : {&bar_k, &bar_v, &bar_s, &bar_done, &bar_raw, &bar_drain})
            mbar_init(smem_u32(b), 1);
        mbar_init(smem_u32(&bar_p), kMathWarps);
        for (int i = 0; i < Sh::kDp; ++i) {
            mbar_init(smem_u32(&bar_dp[i]), 1);
            mbar_init(smem_u32(&bar_ds[i]), kMathWarps);
        }
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(smem_u32(&full_q[i]), 2);  // the tile, and its rows' lse and delta
            mbar_init(smem_u32(&empty_q[i]), 1);
            mbar_init(smem_u32(&full_d[i]), 1);
            mbar_init(smem_u32(&empty_d[i]), 1);
        }
        fence_barrier_init();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // all 512 columns are the block's: their addresses start at 0
    constexpr uint32_t t_s = 0, t_dp = 128, t_dv = t_dp + Sh::kDp * 128, t_dk = t_dv + DP;

    if (items > 0 && warp == kMathWarps + 1) {
        // ---- the producer ----
        const Sequence sq = work.sq;
        int q_first;
        const int per_head = queries_of(sq, work.row0, p.batch.causal, &q_first);
        if (elect_one()) {
            const int64_t key = sq.k0 + work.row0;
            mbar_expect(smem_u32(&bar_k), Sh::kTileBytes);
            load_tile<Sh::kBlocks>(at_k, &map_k, smem_u32(&bar_k), work.khead, key, p.swap_k);
            mbar_expect(smem_u32(&bar_v), Sh::kTileBytes);
            load_tile<Sh::kBlocks>(at_v, &map_v, smem_u32(&bar_v), work.khead, key, p.swap_v);
        }
        __syncwarp();
        int mends = 0, tiles_q = 0, tiles_d = 0;  // tiles brought into the rings
        bool ok = true;
        // one tile of queries (which = 0) or of output gradients (1) into slot `slot`
        const auto bring = [&](bool of_d, uint32_t dst, uint32_t full, int head, int i0) {
            const int valid = sq.n - i0;
            const bool mend = valid < kTileRows && sq.q0 + sq.n < p.batch.tq;
            const uint32_t bar = mend ? smem_u32(&bar_raw) : full;
            if (elect_one()) {
                mbar_expect(bar, Sh::kTileBytes);
                load_tile<Sh::kBlocks>(dst, of_d ? &map_d : &map_q, bar, head, sq.q0 + i0,
                                       of_d ? p.swap_d : p.swap_q);
            }
            __syncwarp();
            if (mend) {
                const int parity = mends++ & 1;
                if (!mbar_wait(bar, parity, &dead)) {
                    mbar_drain(bar, parity);
                    return false;
                }
                zero_rows<Sh::kBlocks>(smem_raw + (dst - smem_u32(smem_raw)), valid);
                fence_async_shared();
                __syncwarp();
                if (elect_one()) mbar_arrive(full);
                __syncwarp();
            }
            return true;
        };
        int head = work.khead * p.group + work.first / per_head;
        int tile = q_first + work.first % per_head;
        for (int i = 0; i < items; ++i) {
            const int slot = i % Sh::kSlots, use = i / Sh::kSlots, i0 = tile * kTileRows;
            if (use > 0) ok = mbar_wait(smem_u32(&empty_q[slot]), (use - 1) & 1, &dead);
            if (!ok) break;
            const uint32_t full = smem_u32(&full_q[slot]);
            ok = bring(false, at_q + slot * Sh::kTileBytes, full, head, i0);
            if (!ok) break;
            const int64_t src = (int64_t)head * p.batch.tq + sq.q0 + i0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = k * 32 + lane;
                rows[slot][0][r] = i0 + r < sq.n ? p.nlse[src + r] : -INFINITY;
                rows[slot][1][r] = i0 + r < sq.n ? p.ndelta[src + r] : 0.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
            ++tiles_q;
            if (use > 0) ok = mbar_wait(smem_u32(&empty_d[slot]), (use - 1) & 1, &dead);
            if (!ok) break;
            ok = bring(true, at_d + slot * Sh::kTileBytes, smem_u32(&full_d[slot]), head, i0);
            if (!ok) break;
            ++tiles_d;
            if (++tile == q_first + per_head) tile = q_first, ++head;
        }
        mbar_drain(smem_u32(&bar_k), 0);
        mbar_drain(smem_u32(&bar_v), 0);
        drain_ring<Sh::kSlots>(full_q, tiles_q);
        drain_ring<Sh::kSlots>(full_d, tiles_d);
    } else if (items > 0 && warp == kMathWarps) {
        // ---- the products ----
        if (elect_one()) {
            constexpr uint32_t word_o = mma_word(128, DP, false, true);
            constexpr uint32_t word_dp = mma_word(128, 128, false, false);
            const uint32_t word_s = word_dp | (p.negative ? kNegateA : 0u);
            bool ok = mbar_wait_one(smem_u32(&bar_k), 0, &dead);
            const auto slot_of = [&](int i) { return i % Sh::kSlots; };
            const auto parity_of = [&](int i) { return (i / Sh::kSlots) & 1; };
            const auto scores = [&](int i) {
                ok = ok && mbar_wait_one(smem_u32(&full_q[slot_of(i)]), parity_of(i), &dead);
                if (!ok) return;
                tmem_fence_after();
                product_columns<DP>(t_s, operand_columns(at_k),
                                    operand_columns(at_q + slot_of(i) * Sh::kTileBytes), word_s,
                                    false);
                mma_commit(smem_u32(&bar_s));
            };
            const auto dprobs = [&](int i) {
                ok = ok && mbar_wait_one(smem_u32(&full_d[slot_of(i)]), parity_of(i), &dead);
                if (!ok) return;
                tmem_fence_after();
                const int at = i % Sh::kDp;
                product_columns<DP>(t_dp + at * 128, operand_columns(at_v),
                                    operand_columns(at_d + slot_of(i) * Sh::kTileBytes), word_dp,
                                    false);
                mma_commit(smem_u32(&bar_dp[at]));
            };
            scores(0);
            ok = ok && mbar_wait_one(smem_u32(&bar_v), 0, &dead);
            dprobs(0);
            for (int i = 0; i < items && ok; ++i) {
                // while the other warps form dS(i): dV, and the next scores
                ok = mbar_wait_one(smem_u32(&bar_p), i & 1, &dead);
                if (!ok) break;
                tmem_fence_after();
                product_rows(t_dv, t_s, 64, operand_rows(at_d + slot_of(i) * Sh::kTileBytes), word_o,
                             i > 0);
                mma_commit(smem_u32(&empty_d[slot_of(i)]));
                if (i + 1 < items) scores(i + 1);
                if (Sh::kDp == 2 && i + 1 < items) dprobs(i + 1);
                // while they form P(i + 1): dK, and the next dO V^T
                ok = ok && mbar_wait_one(smem_u32(&bar_ds[i % Sh::kDp]), (i / Sh::kDp) & 1, &dead);
                if (!ok) break;
                tmem_fence_after();
                product_rows(t_dk, t_dp + i % Sh::kDp * 128, 64, operand_rows(at_q + slot_of(i) * Sh::kTileBytes), word_o,
                             i > 0);
                mma_commit(smem_u32(&empty_q[slot_of(i)]));
                if (Sh::kDp == 1 && i + 1 < items) dprobs(i + 1);
            }
            if (ok) mma_commit(smem_u32(&bar_done));
            mma_commit(smem_u32(&bar_drain));
            mbar_drain(smem_u32(&bar_drain), 0);
        }
    } else if (warp < kMathWarps) {
        // ---- P and dS: one key a thread, half of the tile's queries ----
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_at = t_s + lanes + half * 64;
        const float sl = p.log2_scale;
        const int n = work.sq.n;
        int q_first;
        const int q_end = queries_of(work.sq, work.row0, p.batch.causal, &q_first) + q_first;
        // the first query that sees this thread's key; the last of the tile's keys' first
        const int ahead = work.row0 + n - work.sq.m;
        const int sees = p.batch.causal ? max(0, ahead + r) : 0;
        const int all_see = p.batch.causal ? max(0, ahead + kTileRows - 1) : 0;
        int tile = q_first + (items > 0 ? work.first % (q_end - q_first) : 0);
        for (int i = 0; i < items; ++i) {
            const int slot = i % Sh::kSlots, i0 = tile * kTileRows;
            if (++tile == q_end) tile = q_first;
            const bool masked = i0 < all_see || i0 + kTileRows > n;
            const int lo = sees - i0 - half * 64, hi = n - i0 - half * 64;
            mbar_pass(smem_u32(&full_q[slot]), (i / Sh::kSlots) & 1, &dead);
            mbar_pass(smem_u32(&bar_s), i & 1, &dead);
            tmem_fence_after();
            float pr[64];
            tmem_ld32(reinterpret_cast<uint32_t*>(pr), s_at);
            tmem_ld32(reinterpret_cast<uint32_t*>(pr) + 32, s_at + 32);
            tmem_wait_ld();
            const float4* nl = reinterpret_cast<const float4*>(rows[slot][0] + half * 64);
            const float4* nd = reinterpret_cast<const float4*>(rows[slot][1] + half * 64);
            const float2 sl2 = make_float2(sl, sl);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 v = nl[c >> 2];
                const float2 a = __ffma2_rn(make_float2(pr[c], pr[c + 1]), sl2, make_float2(v.x, v.y));
                const float2 b =
                    __ffma2_rn(make_float2(pr[c + 2], pr[c + 3]), sl2, make_float2(v.z, v.w));
                pr[c] = ex2_approx(a.x);
                pr[c + 1] = ex2_approx(a.y);
                pr[c + 2] = ex2_approx(b.x);
                pr[c + 3] = ex2_approx(b.y);
            }
            if (masked) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c < lo || c >= hi) pr[c] = 0.f;
            }
            store_half(s_at, pr);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_p));
            const uint32_t dp_at = t_dp + i % Sh::kDp * 128 + lanes + half * 64;
            mbar_pass(smem_u32(&bar_dp[i % Sh::kDp]), (i / Sh::kDp) & 1, &dead);
            tmem_fence_after();
            float dp[64];
            tmem_ld32(reinterpret_cast<uint32_t*>(dp), dp_at);
            tmem_ld32(reinterpret_cast<uint32_t*>(dp) + 32, dp_at + 32);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 v = nd[c >> 2];
                const float2 a = __fmul2_rn(
                    make_float2(pr[c], pr[c + 1]),
                    __fadd2_rn(make_float2(dp[c], dp[c + 1]), make_float2(v.x, v.y)));
                const float2 b = __fmul2_rn(
                    make_float2(pr[c + 2], pr[c + 3]),
                    __fadd2_rn(make_float2(dp[c + 2], dp[c + 3]), make_float2(v.z, v.w)));
                dp[c] = a.x, dp[c + 1] = a.y, dp[c + 2] = b.x, dp[c + 3] = b.y;
            }
            if (masked) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c < lo || c >= hi) dp[c] = 0.f;
            }
            store_half(dp_at, dp);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_ds[i % Sh::kDp]));
        }
        if (items > 0) mbar_pass(smem_u32(&bar_done), 0, &dead);
        if (!any_dead(&dead)) {
            tmem_fence_after();
            const int key = work.row0 + r;
            const bool valid = key < work.sq.m, split = work.part >= 0;
            const HeadView& g = half ? p.dk : p.dv;
            __nv_bfloat16* out = valid && !split ? g.row(work.sq.k0 + key, work.khead) : nullptr;
            float* part = valid && split
                              ? p.parts_k + (work.part + r + (half ? 0 : part_rows(p.plan_k))) * DP
                              : nullptr;
            store_row<DP>((half ? t_dk : t_dv) + lanes, out, part, p.dim, half ? p.scale : 1.f,
                          items == 0);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (dead && threadIdx.x == 0) atomicAdd(p.gave_up, 1u);
    if (warp == kMathWarps) {
        __syncwarp();
        tmem_fence_after();
        tmem_free(tmem_at, 512);
    }
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
template <int DP>
struct DqShape {
    static constexpr int kBlocks = DP / kBlockCols;
    static constexpr uint32_t kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kSlotsK = DP == 128 ? 3 : 4, kSlotsV = DP == 128 ? 2 : 4;
    static constexpr uint32_t kSmem = (2 + kSlotsK + kSlotsV) * kTileBytes + 1024;
};

template <int DP>
__device__ __forceinline__ void dq_block(const CUtensorMap& map_q, const CUtensorMap& map_k,
                                         const CUtensorMap& map_v, const CUtensorMap& map_d,
                                         const BwdParams& p, int64_t id) {
    using Sh = DqShape<DP>;
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bar_q, bar_d, bar_s[2], bar_dp, bar_read, bar_ds[2], bar_done, bar_raw,
        bar_drain;
    __shared__ uint64_t full_k[Sh::kSlotsK], empty_k[Sh::kSlotsK], full_v[Sh::kSlotsV],
        empty_v[Sh::kSlotsV];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    __shared__ BwdWork work;
    __shared__ int found;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const bool ok = find_work<false>(p, id, &work);
        if (lane == 0) found = ok, dead = 0;
    }
    __syncthreads();
    if (!found) return;
    const int tiles = work.items;

    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t at_q = smem, at_d = smem + Sh::kTileBytes;
    const uint32_t at_k = smem + 2 * Sh::kTileBytes, at_v = at_k + Sh::kSlotsK * Sh::kTileBytes;
    if (warp == kMathWarps) {
        tmem_alloc(smem_u32(&tmem_at), 512);
    } else if (threadIdx.x == 0) {
        for (uint64_t* b : {&bar_q, &bar_d, &bar_s[0], &bar_s[1], &bar_dp, &bar_done, &bar_raw,
                            &bar_drain})
            mbar_init(smem_u32(b), 1);
        mbar_init(smem_u32(&bar_ds[0]), kMathWarps);
        mbar_init(smem_u32(&bar_ds[1]), kMathWarps);
        mbar_init(smem_u32(&bar_read), kMathWarps);
        for (int i = 0; i < Sh::kSlotsK; ++i) {
            mbar_init(smem_u32(&full_k[i]), 1);
            mbar_init(smem_u32(&empty_k[i]), 1);
        }
        for (int i = 0; i < Sh::kSlotsV; ++i) {
            mbar_init(smem_u32(&full_v[i]), 1);
            mbar_init(smem_u32(&empty_v[i]), 1);
        }
        fence_barrier_init();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // all 512 columns are the block's: their addresses start at 0
    constexpr uint32_t tmem = 0, t_dp = 256, t_dq = 384;

    if (tiles > 0 && warp == kMathWarps + 1) {
        // ---- the producer ----
        const int khead = work.khead, left = work.sq.m - work.first * kTileRows;
        const int64_t k0 = work.sq.k0 + (int64_t)work.first * kTileRows;
        const bool tail = work.sq.k0 + work.sq.m < p.batch.tk;
        if (elect_one()) {
            const int64_t q = work.sq.q0 + work.row0;
            mbar_expect(smem_u32(&bar_q), Sh::kTileBytes);
            load_tile<Sh::kBlocks>(at_q, &map_q, smem_u32(&bar_q), work.head, q, p.swap_q);
            mbar_expect(smem_u32(&bar_d), Sh::kTileBytes);
            load_tile<Sh::kBlocks>(at_d, &map_d, smem_u32(&bar_d), work.head, q, p.swap_d);
        }
        __syncwarp();
        int tiles_k = 0, tiles_v = 0;  // tiles brought into the rings
        bool ok = true;
        for (int j = 0; j < tiles; ++j) {
            const int sk = j % Sh::kSlotsK, uk = j / Sh::kSlotsK;
            const int sv = j % Sh::kSlotsV, uv = j / Sh::kSlotsV;
            const int64_t token = k0 + (int64_t)j * kTileRows;
            if (uk > 0) ok = mbar_wait(smem_u32(&empty_k[sk]), (uk - 1) & 1, &dead);
            if (!ok) break;
            const int valid = left - j * kTileRows;
            const bool mend = valid < kTileRows && tail;
            const uint32_t full = smem_u32(&full_k[sk]), dst = at_k + sk * Sh::kTileBytes;
            const uint32_t bar = mend ? smem_u32(&bar_raw) : full;
            if (elect_one()) {
                mbar_expect(bar, Sh::kTileBytes);
                load_tile<Sh::kBlocks>(dst, &map_k, bar, khead, token, p.swap_k);
            }
            __syncwarp();
            if (mend) {  // once, at the last tile
                ok = mbar_wait(bar, 0, &dead);
                if (!ok) {
                    mbar_drain(bar, 0);
                    break;
                }
                zero_rows<Sh::kBlocks>(smem_raw + (dst - smem_u32(smem_raw)), valid);
                fence_async_shared();
                __syncwarp();
                if (elect_one()) mbar_arrive(full);
                __syncwarp();
            }
            ++tiles_k;
            if (uv > 0) ok = mbar_wait(smem_u32(&empty_v[sv]), (uv - 1) & 1, &dead);
            if (!ok) break;
            if (elect_one()) {
                mbar_expect(smem_u32(&full_v[sv]), Sh::kTileBytes);
                load_tile<Sh::kBlocks>(at_v + sv * Sh::kTileBytes, &map_v, smem_u32(&full_v[sv]),
                                       khead, token, p.swap_v);
            }
            ++tiles_v;
            __syncwarp();
        }
        mbar_drain(smem_u32(&bar_q), 0);
        mbar_drain(smem_u32(&bar_d), 0);
        drain_ring<Sh::kSlotsK>(full_k, tiles_k);
        drain_ring<Sh::kSlotsV>(full_v, tiles_v);
    } else if (tiles > 0 && warp == kMathWarps) {
        // ---- the products ----
        if (elect_one()) {
            constexpr uint32_t word_o = mma_word(128, DP, false, true);
            constexpr uint32_t word_dp = mma_word(128, 128, false, false);
            const uint32_t word_s = word_dp | (p.negative ? kNegateA : 0u);
            bool ok = mbar_wait_one(smem_u32(&bar_q), 0, &dead);
            const auto scores = [&](int j) {
                const int sk = j % Sh::kSlotsK;
                ok = ok && mbar_wait_one(smem_u32(&full_k[sk]), (j / Sh::kSlotsK) & 1, &dead);
                if (!ok) return;
                tmem_fence_after();
                product_columns<DP>(tmem + (j & 1) * 128, operand_columns(at_q),
                                    operand_columns(at_k + sk * Sh::kTileBytes), word_s, false);
                mma_commit(smem_u32(&bar_s[j & 1]));
            };
            const auto dprobs = [&](int j) {
                const int sv = j % Sh::kSlotsV;
                ok = ok && mbar_wait_one(smem_u32(&full_v[sv]), (j / Sh::kSlotsV) & 1, &dead);
                if (!ok) return;
                tmem_fence_after();
                product_columns<DP>(t_dp, operand_columns(at_d),
                                    operand_columns(at_v + sv * Sh::kTileBytes), word_dp, false);
                mma_commit(smem_u32(&bar_dp));
                mma_commit(smem_u32(&empty_v[sv]));
            };
            scores(0);
            ok = ok && mbar_wait_one(smem_u32(&bar_d), 0, &dead);
            dprobs(0);
            if (tiles > 1) scores(1);
            for (int j = 0; j < tiles && ok; ++j) {
                // the next dO V^T as soon as this one is read, while dS(j) is formed from it
                if (j + 1 < tiles) {
                    ok = mbar_wait_one(smem_u32(&bar_read), j & 1, &dead);
                    dprobs(j + 1);
                }
                // dS(j) comes over S(j); two barriers, since dS(j + 1) may follow at once
                ok = ok && mbar_wait_one(smem_u32(&bar_ds[j & 1]), (j >> 1) & 1, &dead);
                if (!ok) break;
                tmem_fence_after();
                const int sk = j % Sh::kSlotsK;
                product_rows(t_dq, tmem + (j & 1) * 128, 64,
                             operand_rows(at_k + sk * Sh::kTileBytes), word_o, j > 0);
                mma_commit(smem_u32(&empty_k[sk]));
                if (j + 2 < tiles) scores(j + 2);
            }
            if (ok) mma_commit(smem_u32(&bar_done));
            mma_commit(smem_u32(&bar_drain));
            mbar_drain(smem_u32(&bar_drain), 0);
        }
    } else if (warp < kMathWarps) {
        // ---- dS: one query a thread, half of the tile's keys ----
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t dp_at = t_dp + lanes + half * 64;
        const float sl = p.log2_scale;
        // keys of this piece that the thread's row sees, and the warp's first row
        const auto limit_of = [&](int row) {
            return seen_keys(work.row0 + row, work.sq.n, work.sq.m, p.batch.causal) -
                   work.first * kTileRows;
        };
        const int limit = limit_of(r), first_limit = limit_of((warp & 3) * 32);
        float nl = -INFINITY, nd = 0.f;
        if (work.row0 + r < work.sq.n) {
            const int64_t at = (int64_t)work.head * p.batch.tq + work.sq.q0 + work.row0 + r;
            nl = p.nlse[at];
            nd = p.ndelta[at];
        }
        const float2 sl2 = make_float2(sl, sl), nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
        for (int j = 0; j < tiles; ++j) {
            const uint32_t s_at = tmem + (j & 1) * 128 + lanes + half * 64;
            mbar_pass(smem_u32(&bar_s[j & 1]), (j >> 1) & 1, &dead);
            tmem_fence_after();
            float pr[64];
            tmem_ld32(reinterpret_cast<uint32_t*>(pr), s_at);
            tmem_ld32(reinterpret_cast<uint32_t*>(pr) + 32, s_at + 32);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                const float2 a = __ffma2_rn(make_float2(pr[c], pr[c + 1]), sl2, nl2);
                pr[c] = ex2_approx(a.x);
                pr[c + 1] = ex2_approx(a.y);
            }
            mbar_pass(smem_u32(&bar_dp), j & 1, &dead);
            tmem_fence_after();
            float dp[64];
            tmem_ld32(reinterpret_cast<uint32_t*>(dp), dp_at);
            tmem_ld32(reinterpret_cast<uint32_t*>(dp) + 32, dp_at + 32);
            tmem_wait_ld();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_read));
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                const float2 a = __fmul2_rn(make_float2(pr[c], pr[c + 1]),
                                            __fadd2_rn(make_float2(dp[c], dp[c + 1]), nd2));
                dp[c] = a.x;
                dp[c + 1] = a.y;
            }
            if ((j + 1) * kTileRows > first_limit) {
                const int left = limit - j * kTileRows - half * 64;
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c >= left) dp[c] = 0.f;
            }
            store_half(s_at, dp);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_ds[j & 1]));
        }
        if (tiles > 0) mbar_pass(smem_u32(&bar_done), 0, &dead);
        if (!any_dead(&dead)) {
            tmem_fence_after();
            const int i = work.row0 + r;
            const bool valid = i < work.sq.n, split = work.part >= 0;
            // each half of the warps writes half of the columns
            const int c0 = half * (DP / 2);
            __nv_bfloat16* out =
                valid && !split ? p.dq.row(work.sq.q0 + i, work.head) + c0 : nullptr;
            float* part = valid && split ? p.parts_q + (work.part + r) * DP + c0 : nullptr;
            store_row<DP / 2>(t_dq + lanes + c0, out, part, p.dim - c0, p.scale, tiles == 0);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (dead && threadIdx.x == 0) atomicAdd(p.gave_up, 1u);
    if (warp == kMathWarps) {
        __syncwarp();
        tmem_fence_after();
        tmem_free(tmem_at, 512);
    }
}

// The blocks of keys, then those of queries.
template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attention_bwd_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ CUtensorMap map_d, const BwdParams p) {
    grid_dep_sync();
    const int64_t of_keys = blocks_of(p.plan_k), id = blockIdx.x;
    if (id < of_keys)
        dkv_block<DP>(map_q, map_k, map_v, map_d, p, id);
    else
        dq_block<DP>(map_q, map_k, map_v, map_d, p, id - of_keys);
}

// The sum of a cut block's pieces, in their order, times the scale, in bfloat16.  DP / 4
// lanes a row; blockIdx.z = 1: dV.
constexpr int kSumThreads = 256;

template <int DP, bool kKeys>
__global__ void __launch_bounds__(kSumThreads) attention_sum_kernel(const BwdParams p) {
    __shared__ Place place;
    __shared__ int found;
    grid_dep_sync();
    const BwdPlan& plan = kKeys ? p.plan_k : p.plan_q;
    if (threadIdx.x < 32) {
        Place at{};
        const bool ok = find_place<kKeys>(p.batch, kTileRows, kKeys ? p.heads_k : p.heads_q,
                                          (int)(plan.whole + blockIdx.x), &at);
        if (threadIdx.x == 0) place = at, found = ok;
    }
    __syncthreads();
    if (!found) return;
    const Sequence sq = place.sq;
    const int row0 = place.tile * kTileRows;
    int unused;
    const int items = kKeys ? queries_of(sq, row0, p.batch.causal, &unused) * p.group
                            : keys_of(sq, row0, p.batch.causal);
    // a piece without work was not begun
    const int pieces = max(1, (items + plan.chunk - 1) / plan.chunk);
    constexpr int kLanes = DP / 4, kRows = kSumThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int rows = min(kTileRows, (kKeys ? sq.m : sq.n) - row0);
    const bool of_v = kKeys && blockIdx.z == 1;
    const float4* parts = reinterpret_cast<const float4*>(
        (kKeys ? p.parts_k : p.parts_q) + (of_v ? part_rows(plan) : 0) * DP);
    const HeadView& g = kKeys ? (of_v ? p.dv : p.dk) : p.dq;
    const float f = of_v ? 1.f : p.scale;
    const int64_t step = plan.rest * plan.slot_rows;  // rows from a piece to the next
    for (int r = blockIdx.y * kRows + threadIdx.x / kLanes; r < rows; r += gridDim.y * kRows) {
        const int64_t at = (int64_t)blockIdx.x * plan.slot_rows + r;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int z = 0; z < pieces; ++z) {
            const float4 v = parts[(z * step + at) * kLanes + lane];
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
        }
        if (lane * 4 < p.dim)
            *reinterpret_cast<uint2*>(g.row((kKeys ? sq.k0 : sq.q0) + row0 + r, place.head) +
                                      lane * 4) =
                make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
    }
}

// Cuts the last wave, or all blocks where they are fewer than the SMs, where a model of the
// waves says that it pays, in units of one tile's time: a block costs its tiles and kStart,
// the sum kSum; less than kGain of the whole is not worth it.  `items`: tiles that the longest
// block may meet.  With the mask or several sequences the short blocks come last, and only
// few blocks are cut.
constexpr int kStart = 4, kSum = 4, kMaxPieces = 16, kLeastChunk = 2;
constexpr double kGain = 0.05;

BwdPlan plan_bwd(int64_t blocks, int64_t items, int64_t tokens, bool uniform) {
    BwdPlan plan{};
    plan.whole = blocks;
    plan.pieces = 1;
    plan.slot_rows = (int)(tokens < kTileRows ? tokens : kTileRows);
    if (!uniform && blocks >= kSms) return plan;
    const auto waves = [](int64_t n) { return (n + kSms - 1) / kSms; };
    const int64_t whole = blocks / kSms * kSms, rest = blocks - whole;
    if (rest == 0) return plan;
    double best = (1.0 - kGain) * (double)(waves(blocks) * (items + kStart));
    for (int cuts = 2; cuts <= kMaxPieces; ++cuts) {
        const int64_t chunk = (items + cuts - 1) / cuts;
        if (chunk < kLeastChunk) break;  // at once where the other side is empty
        const int64_t pieces = (items + chunk - 1) / chunk;
        if (rest * pieces > 4 * kSms) break;
        const double cost = (double)(whole / kSms * (items + kStart) +
                                     waves(rest * pieces) * (chunk + kStart) + kSum);
        if (cost < best) {
            best = cost;
            plan.whole = whole;
            plan.rest = rest;
            plan.chunk = (int)chunk;
            plan.pieces = (int)pieces;
        }
    }
    return plan;
}

int64_t tiles_of(int64_t tokens) { return (tokens + kTileRows - 1) / kTileRows; }

BwdPlan plan_dkv(int64_t tq, int64_t tk, int batch, int heads_q, int heads_k, bool causal) {
    return plan_bwd(tiles_at_most(tk, kTileRows, batch) * heads_k,
                    tiles_of(tq) * (heads_q / heads_k), tk, batch == 1 && !causal);
}
BwdPlan plan_dq(int64_t tq, int64_t tk, int batch, int heads_q, bool causal) {
    return plan_bwd(tiles_at_most(tq, kTileRows, batch) * heads_q, tiles_of(tk), tq,
                    batch == 1 && !causal);
}

struct BwdMaps {
    CUtensorMap q, k, v, d;
};

template <int DP, bool kKeys>
cudaError_t launch_sum(const BwdParams& p, cudaStream_t st) {
    const BwdPlan& plan = kKeys ? p.plan_k : p.plan_q;
    if (plan.pieces <= 1) return cudaSuccess;
    const unsigned rows = kSumThreads / (DP / 4);
    const dim3 grid((unsigned)plan.rest, (plan.slot_rows + 2 * rows - 1) / (2 * rows),
                    kKeys ? 2 : 1);
    return launch(attention_sum_kernel<DP, kKeys>, grid, dim3(kSumThreads), 0, st, p);
}

template <int DP>
cudaError_t launch_dim(const BwdMaps& m, BwdParams p, cudaStream_t st) {
    const Batch& v = p.batch;
    // a side without tokens has no blocks
    if (v.tk > 0) p.plan_k = plan_dkv(v.tq, v.tk, v.batch, p.heads_q, p.heads_k, v.causal);
    if (v.tq > 0) p.plan_q = plan_dq(v.tq, v.tk, v.batch, p.heads_q, v.causal);
    p.parts_q = p.parts_k + 2 * part_rows(p.plan_k) * DP;
    constexpr uint32_t kSmem = std::max(DkvShape<DP>::kSmem, DqShape<DP>::kSmem);
    cudaError_t e = cudaFuncSetAttribute(
        attention_bwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess)
        e = launch(attention_bwd_kernel<DP>,
                   dim3((unsigned)(blocks_of(p.plan_k) + blocks_of(p.plan_q))), dim3(kBwdThreads),
                   kSmem, st, m.q, m.k, m.v, m.d, p);
    if (e == cudaSuccess) e = launch_sum<DP, true>(p, st);
    if (e == cudaSuccess) e = launch_sum<DP, false>(p, st);
    return e;
}

HeadView view(const gs_heads& h) {
    return {static_cast<__nv_bfloat16*>(h.data), h.token_stride, h.head_stride};
}

}  // namespace

// -lse and -delta of every query row, then the pieces of both kinds of blocks
size_t attention_bwd_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads_q,
                                     int heads_k, int head_dim) {
    int64_t rows = 0;
    for (const bool causal : {false, true}) {
        const int64_t a =
            2 * part_rows(plan_dkv(tokens_q, tokens_k, batch, heads_q, heads_k, causal));
        const int64_t b = part_rows(plan_dq(tokens_q, tokens_k, batch, heads_q, causal));
        rows = std::max(rows, a + b);
    }
    return ((size_t)tokens_q * heads_q * 2 * sizeof(float) + 255) / 256 * 256 +
           (size_t)rows * (head_dim <= 64 ? 64 : 128) * sizeof(float);
}

cudaError_t launch_attention_bwd(const gs_attention_shape& s, const gs_heads& q, const gs_heads& k,
                                 const gs_heads& v, const gs_heads& out, const float* lse,
                                 const gs_heads& dout, const gs_heads& dq, const gs_heads& dk,
                                 const gs_heads& dv, const int32_t* cu_q, const int32_t* cu_k,
                                 void* ws, cudaStream_t st) {
    BwdParams p{};
    p.batch = {cu_q, cu_k, s.tokens_q, s.tokens_k, s.batch, s.causal != 0};
    p.heads_q = s.heads_q;
    p.heads_k = s.heads_k;
    p.group = s.heads_q / s.heads_k;
    p.dim = s.head_dim;
    p.negative = s.scale < 0.f;
    p.scale = s.scale;
    p.log2_scale = fabsf(s.scale) * 1.4426950408889634f;
    p.o = view(out);
    p.dout = view(dout);
    p.dq = view(dq);
    p.dk = view(dk);
    p.dv = view(dv);
    p.lse = lse;
    p.nlse = static_cast<float*>(ws);
    p.ndelta = p.nlse + s.tokens_q * s.heads_q;
    p.parts_k = p.nlse + (s.tokens_q * s.heads_q * 2 + 63) / 64 * 64;
    cudaError_t e = gave_up_word(&p.gave_up);
    if (e != cudaSuccess) return e;
    BwdMaps m;
    const auto map = [&](CUtensorMap* out_map, const gs_heads& h, int64_t tokens, int heads,
                         bool* swapped) {
        if (e == cudaSuccess && tokens > 0)
            e = head_map(out_map, h.data, h.token_stride, h.head_stride, tokens, heads, s.head_dim,
                         swapped);
    };
    map(&m.q, q, s.tokens_q, s.heads_q, &p.swap_q);
    map(&m.d, dout, s.tokens_q, s.heads_q, &p.swap_d);
    map(&m.k, k, s.tokens_k, s.heads_k, &p.swap_k);
    map(&m.v, v, s.tokens_k, s.heads_k, &p.swap_v);
    if (s.tokens_q == 0) m.q = m.d = m.k;  // nothing is loaded by them
    if (s.tokens_k == 0) m.k = m.v = m.q;
    if (e != cudaSuccess) return e;
    if (p.batch.tq > 0) {
        const int64_t threads = p.batch.tq * s.heads_q * 16;
        e = launch(attention_delta_kernel,
                   dim3((unsigned)((threads + kDeltaThreads - 1) / kDeltaThreads)),
                   dim3(kDeltaThreads), 0, st, p);
        if (e != cudaSuccess) return e;
    }
    return s.head_dim <= 64 ? launch_dim<64>(m, p, st) : launch_dim<128>(m, p, st);
}

}  // namespace gs
