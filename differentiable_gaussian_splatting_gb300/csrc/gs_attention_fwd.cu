// gs_attention_fwd.cu -- softmax attention, forward, on the tensor cores.
//
//   S = scale Q K^T,  P = exp(S - row maximum),  O = P V / row sum
//
// in one pass over the keys with a running maximum and sum (Milakov and Gimelshein, "Online
// normalizer calculation for softmax", 2018).  A block takes 256 queries of
// one head as two tiles of 128 rows, with the key and value tiles (128 rows) shared by
// both.  A producer warp brings tiles by TMA into a ring, one thread issues the products,
// and four warps per query tile do its softmax, one row a thread: S comes from tensor
// memory, P goes back over it in bfloat16 as the second product's first operand, O stays
// in tensor memory.  While one tile's softmax runs, the tensor cores work on the other's
// products.
//
// What bounds it, at 128 values a head: the tensor cores with the shared memory that feeds
// them.  A 128 x 128 tile takes 1,024 cycles of products; the first product reads both
// operands from shared memory at its full 128 bytes a cycle while TMA writes there too, and
// a tile changes hands twice, so about 1,390 cycles pass (tensor pipe busy 68 % of the
// active time).  16,320 tokens x 16 heads, called one by one: 1,250 us, 1,745 TFLOP/s, 0.94 of
// the rate that the library's matrix product reaches in single calls; back to back, under the
// power limit: 1,340 to 1,375 us from card to card, 0.92 to 0.94 of the library's rate under it.
// At 64 values the handshakes weigh twice as much: 8,160 tokens x 16 heads on 4 in 265 us,
// 1,030 TFLOP/s (243 us without the exponentials, 215 without any softmax: more than half of
// what it stands above its products' 147 is the exchange).  Tried and slower, each against the
// kernel of its time: 16 softmax warps with half a row each (1,260 -> 1,351 us at 16,320 tokens),
// a thread for each query tile's products (1,255 -> 1,326), a whole warp that walks the steps
// (1,283 -> 1,414).
//
// The running maximum is stale on purpose, as in published attention kernels for tensor memory:
// a row's O and sum are rescaled only once its maximum has risen by more than 8 (in powers of
// two), so P stays below 2^8 and the rescaling, which has to wait for the last product, is rare.
//
// P is rounded to bfloat16 for the second product, whose other operand is the caller's bfloat16
// V (both operands of a product have one type, and a product of P's high and low parts would
// double its time); the sum takes the unrounded values in fp32.  By norms the outputs stand
// 0.0020 to 0.0024 from the exact ones, where rounding the exact ones to bfloat16 alone gives
// 0.0016 to 0.0017; exact arithmetic with P rounded gives the same as the kernel.
//
// Where the blocks are fewer than the SMs, or their last wave would be mostly empty, those
// blocks' keys are cut into pieces, a block each, which leave normalised outputs and row
// sums in the workspace for a second kernel to join:
//   lse = ln sum_z exp(lse_z),  O = sum_z exp(lse_z - lse) O_z.
//
// Rows of V beyond the sequence's end are set to zero in shared memory, since their
// probability 0 times what may lie there (another sequence, NaN) is not 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gs_attention.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {
namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kFwdThreads = (kSoftmaxWarps + 2) * 32;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kStale = 8.f;  // powers of two by which a maximum may rise unnoticed

template <int DP>
struct FwdShape {
    static constexpr int kBlocks = DP / kBlockCols;
    static constexpr uint32_t kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kSlots = DP == 128 ? 4 : 8;
    // score tiles in tensor memory beside the two outputs: 512 columns hold 3 or 2
    static constexpr int kScores = DP == 128 ? 2 : 3;
    static constexpr uint32_t kSmem = (2 + kSlots) * kTileBytes + 1024;
};

// How blocks are cut.  Last wave: blocks `whole` .. `whole` + `rest` - 1 are cut into
// `pieces` of `chunk` key tiles, piece by piece.  Spread: all blocks are cut so that kSms
// blocks take them all; since the lengths are on the device, the kernels find the chunk.
constexpr int kSms = 152;
constexpr int kLeastChunk = 4;  // key tiles; below, joining costs more than it saves
struct FwdPlan {
    int64_t whole, rest;
    int chunk, pieces;
    bool spread;
    int slot_rows;  // rows that a piece keeps in the workspace
    __host__ __device__ int64_t part_rows() const {
        return spread ? (int64_t)kSms * slot_rows : pieces > 1 ? pieces * rest * slot_rows : 0;
    }
};

struct FwdParams {
    Batch batch;
    int heads, group, dim;
    bool negative, swap_q, swap_k, swap_v;
    float log2_scale;  // |scale| log2(e)
    HeadView o;
    float* lse;
    unsigned int* gave_up;
    FwdPlan plan;
    float *part_o, *part_lse;  // [pieces][rest][slot_rows][DP], [pieces][rest][slot_rows]
};

// key tiles that query tile t (128 rows) of the block at row0 walks
__device__ __forceinline__ int walked(const Sequence& sq, int row0, int t, bool causal) {
    const int last = min(sq.n, row0 + (t + 1) * kTileRows) - 1;
    return last >= row0 + t * kTileRows
               ? (seen_keys(last, sq.n, sq.m, causal) + kTileRows - 1) / kTileRows
               : 0;
}

// What a block works on, kept in shared memory: registers are short in the softmax.
struct FwdWork {
    Sequence sq;
    int row0;         // first query of the block in its sequence
    int head, khead;
    int key0;         // first key of the block's piece
    int tiles[2];     // key tiles that each of the two query tiles walks
    int64_t part;     // first row in the workspace (-1: the block writes the output itself)
};

// Spread blocks (by one whole warp; lane = sequence): the smallest chunk with which kSms
// blocks suffice, and the place of block or piece `id`.  Pieces of a block are neighbours.
struct Spread {
    int chunk, pieces;  // of the place's sequence
    int piece;          // with `cut`: which one
    int first;          // number of the block's first piece
};

__device__ __forceinline__ bool find_spread(const Batch& v, int heads, int id, bool by_piece,
                                            Place* at, Spread* sp) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    Sequence s{};
    if (lane < v.batch) s = sequence(v, lane);
    const int n = s.n, m = s.m;
    const int blocks = (n + 2 * kTileRows - 1) / (2 * kTileRows) * heads;
    const int keys = (m + kTileRows - 1) / kTileRows;
    int lo = kLeastChunk, hi = max(lo, (int)__reduce_max_sync(all, keys));
    while (lo < hi) {
        const int c = (lo + hi) >> 1;
        if ((int)__reduce_add_sync(all, blocks * max(1, (keys + c - 1) / c)) <= kSms)
            hi = c;
        else
            lo = c + 1;
    }
    const int pieces = max(1, (keys + lo - 1) / lo);
    // blocks (or pieces) up to and with this lane's sequence, and pieces alone
    int sum = by_piece ? blocks * pieces : blocks, sum_p = blocks * pieces;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(all, sum, o), w = __shfl_up_sync(all, sum_p, o);
        if (lane >= o) sum += u, sum_p += w;
    }
    const unsigned hit = __ballot_sync(all, sum > id);
    if (!hit) return false;
    const int l = __ffs(hit) - 1;
    int within = id - (sum - (by_piece ? blocks * pieces : blocks));
    const int piece = by_piece ? within % pieces : 0;
    if (by_piece) within /= pieces;
    const int first = sum_p - blocks * pieces + within * pieces;
    at->b = l;
    at->sq = from_lane(s, l);
    at->head = __shfl_sync(all, within % heads, l);
    at->tile = __shfl_sync(all, within / heads, l);
    sp->chunk = lo;
    sp->pieces = __shfl_sync(all, pieces, l);
    sp->piece = __shfl_sync(all, piece, l);
    sp->first = __shfl_sync(all, first, l);
    return sp->first + sp->pieces <= kSms;  // always, unless offsets overlap
}


template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attention_fwd_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const FwdParams p) {
    using Sh = FwdShape<DP>;
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bar_q[2], bar_s[2 * Sh::kScores], bar_p[2 * Sh::kScores],
        bar_o[2 * Sh::kScores], bar_full[Sh::kSlots],
        bar_empty[Sh::kSlots], bar_raw, bar_drain;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    __shared__ FwdWork work;
    __shared__ int found;

    grid_dep_sync();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        Place at{};
        int piece = 0, chunk = 0;
        int64_t part = -1;
        bool ok;
        if (p.plan.spread) {
            Spread sp;
            ok = find_spread(p.batch, p.heads, blockIdx.x, true, &at, &sp);
            if (ok && sp.pieces > 1) {
                piece = sp.piece;
                chunk = sp.chunk;
                part = (int64_t)blockIdx.x * p.plan.slot_rows;
            }
        } else {
            int64_t id = blockIdx.x;
            if (id >= p.plan.whole) {  // the cut blocks, piece by piece
                piece = (int)((id - p.plan.whole) / p.plan.rest);
                id -= piece * p.plan.rest;
                chunk = p.plan.chunk;
                part = ((int64_t)blockIdx.x - p.plan.whole) * p.plan.slot_rows;
            }
            ok = find_place<false>(p.batch, 2 * kTileRows, p.heads, (int)id, &at);
        }
        if (ok && lane == 0) {
            FwdWork w;
            w.sq = at.sq;
            w.row0 = at.tile * 2 * kTileRows;
            w.head = at.head;
            w.khead = at.head / p.group;
            w.key0 = piece * chunk * kTileRows;
            w.part = part;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                w.tiles[t] = walked(w.sq, w.row0, t, p.batch.causal);
                if (part >= 0) w.tiles[t] = min(max(w.tiles[t] - piece * chunk, 0), chunk);
            }
            if (piece > 0 && w.tiles[0] + w.tiles[1] == 0) ok = false;  // no keys left for it
            work = w;
        }
        if (lane == 0) found = ok, dead = 0;
    }
    __syncthreads();
    if (!found) return;

    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t smem_kv = smem + 2 * Sh::kTileBytes;
    if (warp == kSoftmaxWarps) {
        tmem_alloc(smem_u32(&tmem_at), 512);
    } else if (threadIdx.x == 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bar_q[t]), 1);
        }
        for (int i = 0; i < 2 * Sh::kScores; ++i) {
            mbar_init(smem_u32(&bar_s[i]), 1);
            mbar_init(smem_u32(&bar_p[i]), 4);
            mbar_init(smem_u32(&bar_o[i]), 1);
        }
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(smem_u32(&bar_full[i]), 1);
            mbar_init(smem_u32(&bar_empty[i]), 1);
        }
        mbar_init(smem_u32(&bar_raw), 1);
        mbar_init(smem_u32(&bar_drain), 1);
        fence_barrier_init();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // all 512 columns are the block's: their addresses start at 0
    constexpr uint32_t tmem = 0;
    // The score tiles of the block in their order -- key tile by key tile, first and second
    // query tile in turn as long as each has some -- take the buffers in rotation.
    const auto tmem_s = [&](int x) { return tmem + (x % Sh::kScores) * 128; };
    const auto tmem_o = [&](int t) { return tmem + Sh::kScores * 128 + t * DP; };

    if (warp == kSoftmaxWarps + 1) {
        // ---- the producer: Q, then K and V tiles in turn ----
        const int tiles[2] = {work.tiles[0], work.tiles[1]}, most = max(tiles[0], tiles[1]);
        const int64_t k0 = work.sq.k0 + work.key0;
        const int left = work.sq.m - work.key0, khead = work.khead;
        const bool tail = work.sq.k0 + work.sq.m < p.batch.tk;
        if (most > 0) {
            if (elect_one()) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (tiles[t] > 0) {
                        mbar_expect(smem_u32(&bar_q[t]), Sh::kTileBytes);
                        load_tile<Sh::kBlocks>(smem + t * Sh::kTileBytes, &map_q,
                                               smem_u32(&bar_q[t]), work.head,
                                               work.sq.q0 + work.row0 + t * kTileRows, p.swap_q);
                    }
            }
            __syncwarp();
            int i = 0;  // items issued
            for (; i < 2 * most; ++i) {
                const int slot = i % Sh::kSlots, use = i / Sh::kSlots, j = i >> 1;
                if (use > 0 && !mbar_wait(smem_u32(&bar_empty[slot]), (use - 1) & 1, &dead)) break;
                const uint32_t dst = smem_kv + slot * Sh::kTileBytes;
                const uint32_t full = smem_u32(&bar_full[slot]);
                const bool is_v = i & 1;
                const int valid = left - j * kTileRows;
                // values of another sequence behind this one's end: zeros in their place
                const bool mend = is_v && valid < kTileRows && tail;
                const uint32_t bar = mend ? smem_u32(&bar_raw) : full;
                if (elect_one()) {
                    mbar_expect(bar, Sh::kTileBytes);
                    load_tile<Sh::kBlocks>(dst, is_v ? &map_v : &map_k, bar, khead,
                                           k0 + (int64_t)j * kTileRows,
                                           is_v ? p.swap_v : p.swap_k);
                }
                __syncwarp();
                if (mend) {  // once, at the last tile
                    if (!mbar_wait(bar, 0, &dead)) {
                        mbar_drain(bar, 0);
                        break;
                    }
                    zero_rows<Sh::kBlocks>(smem_raw + (dst - smem_u32(smem_raw)), valid);
                    fence_async_shared();
                    __syncwarp();
                    if (elect_one()) mbar_arrive(full);
                }
                __syncwarp();
            }
            for (int t = 0; t < 2; ++t)
                if (tiles[t] > 0) mbar_drain(smem_u32(&bar_q[t]), 0);
            drain_ring<Sh::kSlots>(bar_full, i);
        }
    } else if (warp == kSoftmaxWarps) {
        // ---- the products ----
        // By one thread (a whole warp that walks the steps with one thread issuing took 1,414
        // us instead of 1,283 on 16,320 tokens x 16 heads x 128).  A step is a key tile and a
        // query tile; scores run kScores steps ahead of the outputs, so that a query tile's
        // softmax finds its next scores ready.
        const int tiles[2] = {work.tiles[0], work.tiles[1]}, most = max(tiles[0], tiles[1]);
        if (most > 0 && elect_one()) {
            constexpr uint32_t word_o = mma_word(128, DP, false, true);
            const uint32_t word_s = mma_word(128, 128, false, false) | (p.negative ? kNegateA : 0u);
            constexpr uint32_t kTileStep = Sh::kTileBytes >> 4;
            const uint32_t op_q = operand_columns(smem), op_k = operand_columns(smem_kv),
                           op_v = operand_rows(smem_kv + Sh::kTileBytes);
            bool ok = true;
            struct Step {
                int j, t;          // key tile, query tile
                int slot, phase;   // of K in the ring, V behind it
                int bar, turn;     // j % kScores and the barrier's phase
                int score;         // score tile
            };
            const auto advance = [&](Step& s) {
                s.score = s.score + 1 == Sh::kScores ? 0 : s.score + 1;
                if (s.t == 0 && tiles[1] > 0) {
                    s.t = 1;
                    return false;
                }
                ++s.j;
                s.t = s.j < tiles[0] ? 0 : 1;
                s.slot += 2;
                if (s.slot == Sh::kSlots) s.slot = 0, s.phase ^= 1;
                if (++s.bar == Sh::kScores) s.bar = 0, s.turn ^= 1;
                return true;  // on to another key tile
            };
            Step ahead{0, tiles[0] > 0 ? 0 : 1, 0, 0, 0, 0, 0}, at = ahead;
            const auto scores = [&]() {
                ok = ok && mbar_wait_one(smem_u32(&bar_full[ahead.slot]), ahead.phase, &dead);
                if (ahead.j == 0) ok = ok && mbar_wait_one(smem_u32(&bar_q[ahead.t]), 0, &dead);
                if (!ok) return;
                tmem_fence_after();
                const Step s = ahead;
                // over a tile of P: products are carried out in the order of their issue
                product_columns<DP>(tmem_s(s.score), op_q + s.t * kTileStep,
                                    op_k + s.slot * kTileStep, word_s, false);
                mma_commit(smem_u32(&bar_s[s.t * Sh::kScores + s.bar]));
                if (advance(ahead)) mma_commit(smem_u32(&bar_empty[s.slot]));
            };
            for (int k = 0; k < Sh::kScores && ahead.j < most; ++k) scores();
            while (at.j < most && ok) {
                ok = mbar_wait_one(smem_u32(&bar_full[at.slot + 1]), at.phase, &dead) &&
                     mbar_wait_one(smem_u32(&bar_p[at.t * Sh::kScores + at.bar]), at.turn, &dead);
                if (!ok) break;
                tmem_fence_after();
                const Step s = at;
                product_rows(tmem_o(s.t), tmem_s(s.score), 32, op_v + s.slot * kTileStep, word_o,
                             s.j > 0);
                mma_commit(smem_u32(&bar_o[s.t * Sh::kScores + s.bar]));
                if (ahead.j < most) scores();
                if (advance(at)) mma_commit(smem_u32(&bar_empty[s.slot + 1]));
            }
            mma_commit(smem_u32(&bar_drain));
            mbar_drain(smem_u32(&bar_drain), 0);
        }
    } else {
        // ---- softmax: one row a thread ----
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's lanes of tensor memory
        // keys of this piece that the thread's row sees, and the warp's first row
        const auto keys_of = [&](int row) {
            return seen_keys(work.row0 + t * kTileRows + row, work.sq.n, work.sq.m,
                             p.batch.causal) - work.key0;
        };
        const int limit = keys_of(r), first_limit = keys_of((warp & 3) * 32);
        const int tiles_t = work.tiles[t];
        // the score tiles go by order(j, t) = steps before (j, t)
        const int tiles_0 = work.tiles[0], tiles_1 = work.tiles[1];
        const float sl = p.log2_scale;
        const uint32_t o_at = tmem_o(t) + lanes;
        // Whether the output has been added to for key tile j.  As for the scores there are
        // kScores barriers in turn: this warp may be that many steps ahead of the outputs, and
        // a barrier's phase can be told from the one before it only.
        const auto output_done = [&](int j) {
            mbar_pass(smem_u32(&bar_o[t * Sh::kScores + j % Sh::kScores]), (j / Sh::kScores) & 1,
                      &dead);
        };
        float top = -INFINITY;
        float2 sum = make_float2(0.f, 0.f);
        for (int j = 0; j < tiles_t; ++j) {
            const uint32_t s_at = tmem_s(min(j + t, tiles_0) + min(j, tiles_1)) + lanes;
            // kScores barriers a query tile: the one of j is used again after P(j) is taken
            mbar_pass(smem_u32(&bar_s[t * Sh::kScores + j % Sh::kScores]), (j / Sh::kScores) & 1,
                      &dead);
            tmem_fence_after();
            uint32_t s[128];
#pragma unroll
            for (int c = 0; c < 128; c += 32) tmem_ld32(s + c, s_at + c);
            tmem_wait_ld();
            if ((j + 1) * kTileRows > first_limit) {  // some row of the warp ends in this tile
                const int left = limit - j * kTileRows;
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (c >= left) s[c] = 0xff800000u;  // -infinity
            }
            float mt[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mt[k] = fmaxf(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
#pragma unroll
            for (int c = 8; c < 128; c += 2)
                mt[(c >> 1) & 3] = max3(mt[(c >> 1) & 3], __uint_as_float(s[c]),
                                        __uint_as_float(s[c + 1]));
            const float high = max3(fmaxf(mt[0], mt[1]), mt[2], mt[3]);
            const bool risen = (high - top) * sl > kStale;
            if (__any_sync(0xffffffffu, risen)) {
                const float f = risen ? ex2_approx((top - high) * sl) : 1.f;
                if (risen) top = high;
                sum.x *= f;
                sum.y *= f;
                if (j > 0) {
                    output_done(j - 1);
                    tmem_fence_after();
#pragma unroll
                    for (int c = 0; c < DP; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o, o_at + c);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st16(o_at + c, o);
                    }
                }
            }
            const float shift = top == -INFINITY ? 0.f : -top * sl;
            const float2 sl2 = make_float2(sl, sl), sh2 = make_float2(shift, shift);
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    float2 x = make_float2(__uint_as_float(s[c + k]), __uint_as_float(s[c + k + 1]));
                    x = __ffma2_rn(x, sl2, sh2);
                    x.x = ex2_approx(x.x);
                    x.y = ex2_approx(x.y);
                    sum = __fadd2_rn(sum, x);
                    w[k >> 1] = pack_bf16(x.x, x.y);
                }
                tmem_st16(s_at + (c >> 1), w);
            }
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_p[t * Sh::kScores + j % Sh::kScores]));
        }
        // ---- the row's output ----
        if (tiles_t > 0) output_done(tiles_t - 1);
        if (!any_dead(&dead)) {
            tmem_fence_after();
            const float l = sum.x + sum.y;
            const int slot_row = t * kTileRows + r, i = work.row0 + slot_row;
            const bool valid = i < work.sq.n, split = work.part >= 0;
            // a row that sees no key (of this piece): zeros
            const bool some = limit > 0 && tiles_t > 0;
            const float f = some ? 1.f / l : 0.f;
            __nv_bfloat16* out = valid && !split ? p.o.row(work.sq.q0 + i, work.head) : nullptr;
            float* out32 = valid && split ? p.part_o + (work.part + slot_row) * DP : nullptr;
#pragma unroll
            for (int c = 0; c < DP; c += 32) {
                uint32_t o[32];
                if (tiles_t > 0) {
                    tmem_ld32(o, o_at + c);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    o[k] = some ? __float_as_uint(__uint_as_float(o[k]) * f) : 0u;
                if (out) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        if (c + k >= p.dim) break;
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16(__uint_as_float(o[k + 2 * e]),
                                             __uint_as_float(o[k + 2 * e + 1]));
                        *reinterpret_cast<uint4*>(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (out32) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<uint4*>(out32 + c + k) =
                            make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                }
            }
            if (valid) {
                // in powers of two until the pieces are joined
                const float lse2 = some ? fmaf(top, sl, log2f(l)) : -INFINITY;
                if (!split)
                    p.lse[(int64_t)work.head * p.batch.tq + work.sq.q0 + i] = lse2 * kLn2;
                else
                    p.part_lse[work.part + slot_row] = lse2;
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (dead && threadIdx.x == 0) atomicAdd(p.gave_up, 1u);
    if (warp == kSoftmaxWarps) {
        __syncwarp();
        tmem_fence_after();
        tmem_free(tmem_at, 512);
    }
}

// A split block's rows from its pieces, in the order of the pieces.  DP / 4 lanes a row.
constexpr int kJoinThreads = 256;

template <int DP>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const FwdParams p) {
    __shared__ Place place;
    __shared__ Spread spread;
    __shared__ int found;
    grid_dep_sync();
    if (threadIdx.x < 32) {
        Place at{};
        Spread sp{p.plan.chunk, p.plan.pieces, 0, (int)blockIdx.x};
        const bool ok = p.plan.spread
                            ? find_spread(p.batch, p.heads, blockIdx.x, false, &at, &sp)
                            : find_place<false>(p.batch, 2 * kTileRows, p.heads,
                                                (int)(p.plan.whole + blockIdx.x), &at);
        if (threadIdx.x == 0) place = at, spread = sp, found = ok && sp.pieces > 1;
    }
    __syncthreads();
    if (!found) return;
    const Sequence sq = place.sq;
    const int row0 = place.tile * 2 * kTileRows;
    constexpr int kLanes = DP / 4;
    const int lane = threadIdx.x % kLanes;
    const int rows = min(2 * kTileRows, sq.n - row0);
    // rows from a piece to the next
    const int64_t step = (p.plan.spread ? 1 : p.plan.rest) * p.plan.slot_rows;
    for (int r = blockIdx.y * (kJoinThreads / kLanes) + threadIdx.x / kLanes; r < rows;
         r += gridDim.y * (kJoinThreads / kLanes)) {
        // a piece without keys for the row's tile was not walked
        const int walks = walked(sq, row0, r / kTileRows, p.batch.causal);
        const int pieces = max(1, (walks + spread.chunk - 1) / spread.chunk);
        const int64_t at = (int64_t)spread.first * p.plan.slot_rows + r;
        float top = -INFINITY;
        bool nan = false;
        for (int z = 0; z < pieces; ++z) {
            const float v = p.part_lse[z * step + at];
            nan |= v != v;
            top = fmaxf(top, v);
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
        if (top != -INFINITY) {
#pragma unroll 4
            for (int z = 0; z < pieces; ++z) {
                const float w = ex2_approx(p.part_lse[z * step + at] - top);
                const float4 v = reinterpret_cast<const float4*>(p.part_o)[(z * step + at) * kLanes + lane];
                sum += w;
                o.x = fmaf(w, v.x, o.x);
                o.y = fmaf(w, v.y, o.y);
                o.z = fmaf(w, v.z, o.z);
                o.w = fmaf(w, v.w, o.w);
            }
        }
        const float f = nan ? NAN : (sum > 0.f ? 1.f / sum : 0.f);
        const int64_t token = sq.q0 + row0 + r;
        if (lane * 4 < p.dim)
            *reinterpret_cast<uint2*>(p.o.row(token, place.head) + lane * 4) =
                make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
        if (lane == 0)
            p.lse[(int64_t)place.head * p.batch.tq + token] =
                nan ? NAN : (sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY);
    }
}

// The last wave is cut where a model of the waves says that it pays, in units of one key
// tile's time: a block costs its tiles and kStart for its start and end, the join kJoin, and
// less than kGain of the whole is not worth it (at 8,160 tokens x 16 heads x 128 cutting
// 56 blocks of 512 took 380 -> 362 us; at 16,320 tokens, 112 of 1,024, 1,267 -> 1,274 us).
constexpr int kStart = 3, kJoin = 4, kMaxPieces = 16;
constexpr double kGain = 0.05;

FwdPlan plan_fwd(int64_t tq, int64_t tk, int batch, int heads, bool causal) {
    const int rows = 2 * kTileRows;
    const int64_t blocks = tiles_at_most(tq, rows, batch) * heads;
    const int64_t keys = (tk + kTileRows - 1) / kTileRows;
    FwdPlan plan{};
    plan.whole = blocks;
    plan.pieces = 1;
    plan.slot_rows = (int)(tq < rows ? tq : rows);
    if (blocks < kSms) {
        plan.spread = batch <= 32 && keys > kLeastChunk;
        return plan;
    }
    // under the mask, or with sequences of several lengths, the short blocks come last
    if (causal || batch > 1) return plan;
    const auto waves = [](int64_t n) { return (n + kSms - 1) / kSms; };
    const int64_t whole = blocks / kSms * kSms, rest = blocks - whole;
    if (rest == 0) return plan;
    double best = (1.0 - kGain) * (double)(waves(blocks) * (keys + kStart));
    for (int cuts = 2; cuts <= kMaxPieces; ++cuts) {
        const int64_t chunk = (keys + cuts - 1) / cuts;
        if (chunk < kLeastChunk) break;  // at once without keys
        const int64_t pieces = (keys + chunk - 1) / chunk;
        const double cost = (double)(whole / kSms * (keys + kStart) +
                                     waves(rest * pieces) * (chunk + kStart) + kJoin);
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

template <int DP>
cudaError_t launch_dim(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       const FwdParams& p, cudaStream_t st) {
    cudaError_t e =
        cudaFuncSetAttribute(attention_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)FwdShape<DP>::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = p.plan.spread ? kSms : p.plan.whole + p.plan.rest * p.plan.pieces;
    e = launch(attention_fwd_kernel<DP>, dim3((unsigned)blocks), dim3(kFwdThreads),
               FwdShape<DP>::kSmem, st, mq, mk, mv, p);
    if (e != cudaSuccess || (!p.plan.spread && p.plan.pieces == 1)) return e;
    const int rows = kJoinThreads / (DP / 4);
    const unsigned y = (unsigned)((p.plan.slot_rows + 4 * rows - 1) / (4 * rows));
    const int64_t joined = p.plan.spread ? p.plan.whole : p.plan.rest;
    return launch(attention_join_kernel<DP>, dim3((unsigned)joined, y), dim3(kJoinThreads), 0, st,
                  p);
}

}  // namespace

size_t attention_fwd_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads,
                                     int head_dim) {
    // whatever the mask
    const int64_t a = plan_fwd(tokens_q, tokens_k, batch, heads, false).part_rows();
    const int64_t b = plan_fwd(tokens_q, tokens_k, batch, heads, true).part_rows();
    const int64_t rows = a > b ? a : b;
    return (size_t)rows * ((head_dim <= 64 ? 64 : 128) + 1) * sizeof(float);
}

cudaError_t launch_attention_fwd(const gs_attention_shape& s, const gs_heads& q, const gs_heads& k,
                                 const gs_heads& v, const gs_heads& out, float* lse,
                                 const int32_t* cu_q, const int32_t* cu_k, void* ws,
                                 cudaStream_t st) {
    FwdParams p{};
    p.batch = {cu_q, cu_k, s.tokens_q, s.tokens_k, s.batch, s.causal != 0};
    p.heads = s.heads_q;
    p.group = s.heads_q / s.heads_k;
    p.dim = s.head_dim;
    p.negative = s.scale < 0.f;
    // a zero scale as one too small to matter: masked scores of -infinity stay defined
    p.log2_scale = fmaxf(fabsf(s.scale) * 1.4426950408889634f, 1e-30f);
    p.o = {static_cast<__nv_bfloat16*>(out.data), out.token_stride, out.head_stride};
    p.lse = lse;
    p.plan = plan_fwd(s.tokens_q, s.tokens_k, s.batch, s.heads_q, s.causal != 0);
    p.part_o = static_cast<float*>(ws);
    p.part_lse = p.part_o + p.plan.part_rows() * (s.head_dim <= 64 ? 64 : 128);
    CUtensorMap mq, mk, mv;
    cudaError_t e = gave_up_word(&p.gave_up);
    if (e != cudaSuccess) return e;
    e = head_map(&mq, q.data, q.token_stride, q.head_stride, s.tokens_q, s.heads_q,
                             s.head_dim, &p.swap_q);
    mk = mv = mq;  // without keys nothing is loaded by them
    if (e == cudaSuccess && s.tokens_k > 0) {
        e = head_map(&mk, k.data, k.token_stride, k.head_stride, s.tokens_k, s.heads_k, s.head_dim,
                     &p.swap_k);
        if (e == cudaSuccess)
            e = head_map(&mv, v.data, v.token_stride, v.head_stride, s.tokens_k, s.heads_k,
                         s.head_dim, &p.swap_v);
    }
    if (e != cudaSuccess) return e;
    return s.head_dim <= 64 ? launch_dim<64>(mq, mk, mv, p, st) : launch_dim<128>(mq, mk, mv, p, st);
}

}  // namespace gs
