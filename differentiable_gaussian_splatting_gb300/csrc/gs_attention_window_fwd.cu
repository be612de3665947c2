// gs_attention_window_fwd.cu -- attention over a window of keys and the first few (sinks), forward,
// on the tensor cores.  Formulas, tiles and roundings are those of gs_attention_fwd.cu; what differs
// is that a block of 256 queries meets few keys.
//
// A block walks the tiles of its window and, where that begins behind it, tile 0 for the sinks.  The
// second of its two query tiles leaves out the tile that only the first one sees.  Where the sinks
// are at most kSinkCols, their tile's products and softmax are kSinkCols wide.
//
// With 10 key tiles a block's start and end (place, loads, first product and softmax, the output's
// way to memory) would take as long as its products, so the blocks of an SM follow each other
// without a gap: one CTA an SM goes through its share of them.  A planner warp finds the places ahead
// of time, a producer warp brings the tiles, one thread issues the products, eight warps do the
// softmax; a ring of descriptions (WindowWork) takes them from block to block, each at its own pace.
// The rings of tiles, score tiles and barriers run on through all blocks.
//
// Measured: 16,320 tokens, 16 heads on 4 x 128, 1,024 keys and 4 sinks: 138 us, 965 TFLOP/s of the
// pairs that are seen; 10.2 steps of 1.5 us a block (a key tile for both query tiles, the rate of
// gs_attention_fwd.cu) and 4 us of its end, during which its softmax warps do nothing else.  One block a
// CTA took 162 us.  4,346 + 2,500 + 64 + 1 + 1,039 tokens, 8 heads x 64, 513 keys: 26.4 us, of which two
// rounds of blocks on every SM take 22.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gs_attention_fwd.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {
namespace {

constexpr int kProductWarp = kSoftmaxWarps, kProducerWarp = kProductWarp + 1,
              kPlannerWarp = kProducerWarp + 1;
constexpr int kWindowThreads = (kPlannerWarp + 2) * 32;  // whole groups of four warps
// Registers of the softmax warps' groups and of the last one: as many in all as at launch.  (With 216
// and 72 as fast, with 232 and 40 159 us instead of 138 at 16,320 tokens.  Four warps more that write
// the outputs meanwhile leave the softmax warps 184, 176 or 168: 152, 157 and 163 us.)
constexpr int kSoftmaxRegisters = 208, kOtherRegisters = 88;
static_assert(2 * kSoftmaxRegisters + kOtherRegisters == 3 * kLaunchRegisters, "the launch's");
constexpr int kWorks = 6;      // descriptions in flight: more than scores may be blocks ahead
constexpr int kStageBytes = 32 * 64;  // a warp's: 32 rows of 32 values on their way to memory
constexpr int kSinkCols = 32;  // columns of the sinks' narrow tile
// who lets go of a description: the softmax warps, the producer and the thread of the products
constexpr int kReaders = kSoftmaxWarps + 2;

// A block: a piece of the key tiles that 256 queries of a head walk.
struct WindowWork {
    Sequence sq;
    int row0;         // first query of the block in its sequence
    int head, khead;
    int64_t part;     // first row in the workspace (-1: the block writes the output itself)
    Walk walk;        // steps are those of the walk from `step0` on
    int step0;
    int end[2];       // each query tile's end among the steps
    int skip;         // the step that the second query tile leaves out (-1: none)
    int narrow;       // steps before this one are the sinks' narrow tile
    bool last;        // no block: the end
};

__device__ __forceinline__ int steps_of(const WindowWork& w) { return max(w.end[0], w.end[1]); }
// how many steps query tile t takes
__device__ __forceinline__ int tiles_of(const WindowWork& w, int t) {
    return w.end[t] - (t == 1 && w.skip >= 0 ? 1 : 0);
}

// By one whole warp: block `id`, or false where there is none.
__device__ __forceinline__ bool find_work(const FwdParams& p, int64_t id, WindowWork* w) {
    Place at{};
    int piece = 0, chunk = 0;
    w->part = -1;
    if (p.plan.spread) {
        Spread sp;
        if (!find_spread(p.batch, p.heads, (int)id, true, p.plan.most_keys, &at, &sp)) return false;
        if (sp.pieces > 1) {
            piece = sp.piece;
            chunk = sp.chunk;
            w->part = id * p.plan.slot_rows;
        }
    } else if (!find_place<false>(p.batch, 2 * kTileRows, p.heads, (int)id, &at)) {
        return false;
    }
    w->sq = at.sq;
    w->row0 = at.tile * 2 * kTileRows;
    w->head = at.head;
    w->khead = at.head / p.group;
    w->last = false;
    const FwdWalk f = walk_of_block(p.window, w->sq, w->row0);
    w->walk = f.walk;
    w->step0 = 0;
    w->end[0] = f.end[0];
    w->end[1] = f.end[1];
    w->skip = f.skip;
    if (w->part >= 0) {
        w->step0 = piece * chunk;
        for (int t = 0; t < 2; ++t) w->end[t] = min(max(f.end[t] - w->step0, 0), chunk);
        w->skip = f.skip >= w->step0 ? f.skip - w->step0 : -1;
    }
    if (w->skip >= w->end[1]) w->skip = -1;
    if (w->skip >= 0 && w->skip == w->end[1] - 1) --w->end[1], w->skip = -1;  // a piece's last
    w->narrow = p.window.sinks <= kSinkCols ? max(0, f.walk.extra - w->step0) : 0;
    return piece == 0 || steps_of(*w) > 0;  // a piece without keys has nothing to do
}

// By one whole warp: zeros and -infinity for the rows of a block that sees no key.
__device__ __forceinline__ void write_nothing(const FwdParams& p, const WindowWork& w, int dp) {
    const int lane = threadIdx.x & 31, rows = min(2 * kTileRows, w.sq.n - w.row0);
    const bool split = w.part >= 0;
    const int words = split ? dp / 4 : p.dim / 8;  // of 16 bytes in a row
    for (int i = lane; i < rows * words; i += 32) {
        const int r = i / words, c = i - r * words;
        uint4* row = split ? reinterpret_cast<uint4*>(p.part_o + (w.part + r) * dp)
                           : reinterpret_cast<uint4*>(p.o.row(w.sq.q0 + w.row0 + r, w.head));
        row[c] = make_uint4(0, 0, 0, 0);
    }
    float* lse = split ? p.part_lse + w.part
                       : p.lse + (int64_t)w.head * p.batch.tq + w.sq.q0 + w.row0;
    for (int r = lane; r < rows; r += 32) lse[r] = -INFINITY;
}

// A softmax row's running maximum and sum.
struct RowState {
    float top;
    float2 sum;
};

// One step of a row: kCols scores to probabilities, over themselves; the output is rescaled where
// the maximum has risen.  `visible`: whether all columns are seen by the warp's rows;
// `output_done` waits for the products that the output holds (any: there are some).
template <int DP, int kCols, typename Done>
__device__ __forceinline__ void softmax_step(RowState& row, uint32_t s_at, uint32_t o_at, float sl,
                                             bool visible, int lo, int hi, int sinks, bool any,
                                             const Done& output_done) {
    uint32_t s[kCols];
#pragma unroll
    for (int c = 0; c < kCols; c += 32) tmem_ld32(s + c, s_at + c);
    tmem_wait_ld();
    if (!visible) {
#pragma unroll
        for (int c = 0; c < kCols; c += 32)
            mask_by_bits(s + c, seen_bits(lo - c, hi - c, sinks - c), 0xff800000u);  // -infinity
    }
    float mt[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        mt[k] = fmaxf(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
#pragma unroll
    for (int c = 8; c < kCols; c += 2)
        mt[(c >> 1) & 3] =
            max3(mt[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    const float high = max3(fmaxf(mt[0], mt[1]), mt[2], mt[3]);
    const bool risen = (high - row.top) * sl > kStale;
    if (__any_sync(0xffffffffu, risen)) {
        const float f = risen ? ex2_approx((row.top - high) * sl) : 1.f;
        if (risen) row.top = high;
        row.sum.x *= f;
        row.sum.y *= f;
        if (any) {
            output_done();
            tmem_fence_after();
#pragma unroll
            for (int c = 0; c < DP; c += 16) {
                uint32_t o[16];
                tmem_ld16(o, o_at + c);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st16(o_at + c, o);
            }
        }
    }
    const float shift = row.top == -INFINITY ? 0.f : -row.top * sl;
    const float2 sl2 = make_float2(sl, sl), sh2 = make_float2(shift, shift);
#pragma unroll
    for (int c = 0; c < kCols; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float2 x = make_float2(__uint_as_float(s[c + k]), __uint_as_float(s[c + k + 1]));
            x = __ffma2_rn(x, sl2, sh2);
            x.x = ex2_approx(x.x);
            x.y = ex2_approx(x.y);
            row.sum = __fadd2_rn(row.sum, x);
            w[k >> 1] = pack_bf16(x.x, x.y);
        }
        tmem_st16(s_at + (c >> 1), w);
    }
    tmem_wait_st();
    tmem_fence_before();
}

template <int DP>
__global__ void __launch_bounds__(kWindowThreads, 1)
    attention_window_fwd_kernel(const __grid_constant__ CUtensorMap map_q,
                                const __grid_constant__ CUtensorMap map_k,
                                const __grid_constant__ CUtensorMap map_v, const FwdParams p,
                                int64_t blocks) {
    using Sh = FwdShape<DP>;
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bar_q[2], bar_q_free[2], bar_s[2 * Sh::kScores], bar_p[2 * Sh::kScores],
        bar_o[2 * Sh::kScores], bar_full[Sh::kSlots], bar_empty[Sh::kSlots], bar_raw, bar_drain,
        bar_work[kWorks], bar_work_free[kWorks];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    __shared__ WindowWork works[kWorks];

    grid_dep_sync();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t smem_kv = smem + 2 * Sh::kTileBytes;
    if (warp == kProductWarp) {
        tmem_alloc(smem_u32(&tmem_at), 512);
    } else if (threadIdx.x == 0) {
        dead = 0;
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bar_q[t]), 1);
            mbar_init(smem_u32(&bar_q_free[t]), 1);
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
        for (int i = 0; i < kWorks; ++i) {
            mbar_init(smem_u32(&bar_work[i]), 1);
            mbar_init(smem_u32(&bar_work_free[i]), kReaders);
        }
        mbar_init(smem_u32(&bar_raw), 1);
        mbar_init(smem_u32(&bar_drain), 1);
        fence_barrier_init();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // all 512 columns are the CTA's: their addresses start at 0
    constexpr uint32_t tmem = 0;
    // The score tiles of all blocks in their order -- key tile by key tile, first and second
    // query tile in turn where they take the step -- take the buffers in rotation.
    const auto tmem_s = [&](int x) { return tmem + x * 128; };
    const auto tmem_o = [&](int t) { return tmem + Sh::kScores * 128 + t * DP; };

    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegisters));
        // ---- softmax: one row a thread ----
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's lanes of tensor memory
        const float sl = p.log2_scale;
        const uint32_t o_at = tmem_o(t) + lanes;
        char* stage = smem_raw + (smem + FwdShape<DP>::kSmem - 1024 - smem_u32(smem_raw)) +
                      warp * kStageBytes;
        int base = 0;   // score tile of the block's first step
        int steps = 0;  // of this query tile, of all blocks
        // Whether the output has been added to for this query tile's step i.  As for the scores
        // there are kScores barriers in turn: this warp may be that many steps ahead of the outputs,
        // and a barrier's phase can be told from the one before it only.
        const auto output_done = [&](int i) {
            mbar_pass(smem_u32(&bar_o[t * Sh::kScores + i % Sh::kScores]), (i / Sh::kScores) & 1,
                      &dead);
        };
        for (int n = 0;; ++n) {
            const int at = n % kWorks;
            if (!mbar_wait(smem_u32(&bar_work[at]), (n / kWorks) & 1, &dead)) break;
            const WindowWork& w = works[at];
            if (w.last) break;
            const int tiles_0 = tiles_of(w, 0), tiles_1 = tiles_of(w, 1);
            const int tiles_t = t == 0 ? tiles_0 : tiles_1, skip = w.skip;
            const int row = w.row0 + t * kTileRows + r;
            // what the row sees, the end of the warp's first row's keys and the start of its last
            // one's
            const Seen see = seen_by(p.window, row, w.sq.n, w.sq.m);
            const int first_hi = __shfl_sync(0xffffffffu, see.hi, 0);
            const int last_lo = __shfl_sync(0xffffffffu, see.lo, 31);
            RowState state{-INFINITY, make_float2(0.f, 0.f)};
            for (int j = 0; j < tiles_t; ++j, ++steps) {
                // key tile of the block's order, and the score tiles before this one
                const int v = t == 1 && skip >= 0 && j >= skip ? j + 1 : j;
                const int before = t == 1 ? min(v + 1, tiles_0) + j
                                          : j + min(j - (skip >= 0 && j > skip ? 1 : 0), tiles_1);
                const uint32_t s_at = tmem_s((base + before) % Sh::kScores) + lanes;
                const int key = w.walk.tile(w.step0 + v) * kTileRows;
                // kScores barriers a query tile: the one of a step is used again after its P is taken
                mbar_pass(smem_u32(&bar_s[t * Sh::kScores + steps % Sh::kScores]),
                          (steps / Sh::kScores) & 1, &dead);
                tmem_fence_after();
                const auto done = [&]() { output_done(steps - 1); };
                if (v < w.narrow)
                    softmax_step<DP, kSinkCols>(state, s_at, o_at, sl, false, see.lo, see.hi,
                                                see.sinks, j > 0, done);
                else
                    softmax_step<DP, kTileRows>(state, s_at, o_at, sl,
                                                key + kTileRows <= first_hi && key >= last_lo,
                                                see.lo - key, see.hi - key, see.sinks - key, j > 0,
                                                done);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&bar_p[t * Sh::kScores + steps % Sh::kScores]));
            }
            base = (base + tiles_0 + tiles_1) % Sh::kScores;
            // ---- the row's output ----
            if (tiles_t > 0) output_done(steps - 1);
            if (any_dead(&dead)) break;
            tmem_fence_after();
            const float l = state.sum.x + state.sum.y;
            const int64_t part = w.part;
            const int64_t token = w.sq.q0 + row;
            const bool valid = row < w.sq.n, split = part >= 0;
            // a row that sees no key (of this piece): zeros
            const bool some = tiles_t > 0 && l != 0.f;
            const float f = some ? 1.f / l : 0.f;
            float* out32 =
                valid && split ? p.part_o + (part + t * kTileRows + r) * DP : nullptr;
            // the warp's first row, and how many it has
            const int rows = split ? 0 : w.sq.n - (row - lane);
            __nv_bfloat16* out = p.o.row(token - lane, w.head);
            if (valid) {
                // in powers of two until the pieces are joined
                const float lse2 = some ? fmaf(state.top, sl, log2f(l)) : -INFINITY;
                if (!split)
                    p.lse[(int64_t)w.head * p.batch.tq + token] = lse2 * kLn2;
                else
                    p.part_lse[part + t * kTileRows + r] = lse2;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_work_free[at]));
            const float2 f2 = make_float2(f, f);
            // 32 columns of the row, normalised
            const auto columns = [&](float2 (&o)[16], int c) {
                if (tiles_t > 0) {
                    tmem_ld32(reinterpret_cast<uint32_t*>(o), o_at + c);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __fmul2_rn(o[k], f2);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = make_float2(0.f, 0.f);
                }
            };
            if (!split) {
                // Through shared memory, so that a store takes 64 bytes of 8 rows instead of 16 of 32.
                // A row's 16-byte words change places by its number: no two lanes meet in a bank.
                const int first = lane >> 2, turn = lane >> 1 & 3;
                char* put = stage + lane * 64;
                const char* get = stage + first * 64 + ((lane & 3) ^ (first >> 1 & 3)) * 16;
                __nv_bfloat16* to = out + first * p.o.ts + (lane & 3) * 8;
#pragma unroll
                for (int c = 0; c < DP; c += 32) {
                    float2 o[16];
                    columns(o, c);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4*>(put + (k ^ turn) * 16) = make_uint4(
                            pack_bf16(o[4 * k].x, o[4 * k].y), pack_bf16(o[4 * k + 1].x, o[4 * k + 1].y),
                            pack_bf16(o[4 * k + 2].x, o[4 * k + 2].y),
                            pack_bf16(o[4 * k + 3].x, o[4 * k + 3].y));
                    __syncwarp();
                    if (c + (lane & 3) * 8 < p.dim)
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // eight rows on, a row's words lie as here
                            if (k * 8 + first < rows)
                                *reinterpret_cast<uint4*>(to + k * 8 * p.o.ts + c) =
                                    *reinterpret_cast<const uint4*>(get + k * 8 * 64);
                    __syncwarp();
                }
            } else {
#pragma unroll
                for (int c = 0; c < DP; c += 32) {
                    float2 o[16];
                    columns(o, c);
                    if (out32)
#pragma unroll
                        for (int k = 0; k < 16; k += 2)
                            *reinterpret_cast<float4*>(out32 + c + 2 * k) =
                                make_float4(o[k].x, o[k].y, o[k + 1].x, o[k + 1].y);
                }
            }
            tmem_fence_before();  // the output may be written over once the next P is there
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegisters));
        if (warp == kPlannerWarp) {
            // ---- the planner ----
            int n = 0;  // descriptions so far
            for (int64_t id = blockIdx.x;; id += gridDim.x) {
                WindowWork w;
                const bool end = id >= blocks;
                if (!end) {
                    if (!find_work(p, id, &w)) continue;
                    if (steps_of(w) == 0) {
                        write_nothing(p, w, DP);
                        continue;
                    }
                }
                const int slot = n % kWorks, use = n / kWorks;
                if (use > 0 && !mbar_wait_block(smem_u32(&bar_work_free[slot]), (use - 1) & 1, &dead))
                    break;
                w.last = end;
                if (lane == 0) {
                    works[slot] = w;
                    mbar_arrive(smem_u32(&bar_work[slot]));
                }
                __syncwarp();
                ++n;
                if (end) break;
            }
        } else if (warp == kProducerWarp) {
            // ---- the producer: Q, then K and V tiles in turn ----
            int items = 0, mends = 0;  // tiles issued into the ring; those mended
            int loads[2] = {0, 0};     // of Q
            bool ok = true;
            for (int n = 0; ok; ++n) {
                const int at = n % kWorks;
                if (!mbar_wait(smem_u32(&bar_work[at]), (n / kWorks) & 1, &dead)) break;
                const WindowWork& w = works[at];
                if (w.last) break;
                const int steps = steps_of(w);
                const int64_t q0 = w.sq.q0 + w.row0, k0 = w.sq.k0;
                const int head = w.head, khead = w.khead, m = w.sq.m, step0 = w.step0;
                const Walk walk = w.walk;
                const bool tail = k0 + m < p.batch.tk;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || tiles_of(w, t) == 0) continue;
                    // once the last block's scores of this query tile are formed
                    if (loads[t] > 0)
                        ok = mbar_wait(smem_u32(&bar_q_free[t]), (loads[t] - 1) & 1, &dead);
                    if (!ok) continue;
                    if (elect_one()) {
                        mbar_expect(smem_u32(&bar_q[t]), Sh::kTileBytes);
                        load_tile<Sh::kBlocks>(smem + t * Sh::kTileBytes, &map_q, smem_u32(&bar_q[t]),
                                               head, q0 + t * kTileRows, p.swap_q);
                    }
                    __syncwarp();
                    ++loads[t];
                }
                if (lane == 0) mbar_arrive(smem_u32(&bar_work_free[at]));
                for (int i = 0; i < 2 * steps && ok; ++i) {
                    const int slot = items % Sh::kSlots, use = items / Sh::kSlots;
                    const int tile = walk.tile(step0 + (i >> 1));
                    ok = use == 0 || mbar_wait(smem_u32(&bar_empty[slot]), (use - 1) & 1, &dead);
                    if (!ok) break;
                    const uint32_t dst = smem_kv + slot * Sh::kTileBytes;
                    const uint32_t full = smem_u32(&bar_full[slot]);
                    const bool is_v = i & 1;
                    const int valid = m - tile * kTileRows;
                    // values of another sequence behind this one's end: zeros in their place
                    const bool mend = is_v && valid < kTileRows && tail;
                    const uint32_t bar = mend ? smem_u32(&bar_raw) : full;
                    if (elect_one()) {
                        mbar_expect(bar, Sh::kTileBytes);
                        load_tile<Sh::kBlocks>(dst, is_v ? &map_v : &map_k, bar, khead,
                                               k0 + (int64_t)tile * kTileRows,
                                               is_v ? p.swap_v : p.swap_k);
                    }
                    __syncwarp();
                    if (mend) {
                        const int parity = mends++ & 1;
                        ok = mbar_wait(bar, parity, &dead);
                        if (!ok) {
                            mbar_drain(bar, parity);
                            break;
                        }
                        zero_rows<Sh::kBlocks>(smem_raw + (dst - smem_u32(smem_raw)), valid);
                        fence_async_shared();
                        __syncwarp();
                        if (elect_one()) mbar_arrive(full);
                    }
                    __syncwarp();
                    ++items;
                }
            }
            for (int t = 0; t < 2; ++t)
                if (loads[t] > 0) mbar_drain(smem_u32(&bar_q[t]), (loads[t] - 1) & 1);
            drain_ring<Sh::kSlots>(bar_full, items);
        } else if (warp == kProductWarp) {
            // ---- the products ----
            // By one thread.  A step is a key tile and a query tile; scores run kScores steps ahead of
            // the outputs, across blocks too, so that a query tile's softmax finds its next scores
            // ready.
            if (elect_one()) {
                constexpr uint32_t word_o = mma_word(128, DP, false, true);
                const uint32_t sign = p.negative ? kNegateA : 0u;
                const uint32_t word_s = mma_word(128, 128, false, false) | sign;
                const uint32_t word_sinks = mma_word(128, kSinkCols, false, false) | sign;
                constexpr uint32_t kTileStep = Sh::kTileBytes >> 4;
                const uint32_t op_q = operand_columns(smem), op_k = operand_columns(smem_kv),
                               op_v = operand_rows(smem_kv + Sh::kTileBytes);
                bool ok = true;
                // A place in the order of steps.  Rings and barriers run on from block to block.
                struct Cursor {
                    int n;                           // block
                    bool in;                         // whether its description has been read:
                    int end0, end1, skip, narrow;
                    int j, t;                        // step, query tile
                    bool begun0, begun1;             // query tile t has had a step
                    int slot, phase;                 // of K in the ring, V behind it
                    int bar0, turn0, bar1, turn1;    // of each query tile's steps: barrier and phase
                    int score;                       // score tile
                };
                const auto enter = [&](Cursor& c) {  // false: no more blocks
                    const int i = c.n % kWorks;
                    ok = ok && mbar_wait_one(smem_u32(&bar_work[i]), (c.n / kWorks) & 1, &dead);
                    if (!ok || works[i].last) return false;
                    c.in = true;
                    c.end0 = works[i].end[0];
                    c.end1 = works[i].end[1];
                    c.skip = works[i].skip;
                    c.narrow = works[i].narrow;
                    c.j = 0;
                    c.t = c.end0 > 0 ? 0 : 1;
                    c.begun0 = c.begun1 = false;
                    return true;
                };
                const auto bar_of = [&](const Cursor& c) {
                    return c.t == 0 ? c.bar0 : Sh::kScores + c.bar1;
                };
                // whether no step before took the key tile: it may still be on its way
                const auto first_of_tile = [&](const Cursor& c) { return c.t == 0 || c.j >= c.end0; };
                const auto move = [&](Cursor& c) {  // true: the key tile is left
                    if (++c.score == Sh::kScores) c.score = 0;
                    if (c.t == 0) {
                        c.begun0 = true;
                        if (++c.bar0 == Sh::kScores) c.bar0 = 0, c.turn0 ^= 1;
                        if (c.j < c.end1 && c.j != c.skip) {
                            c.t = 1;
                            return false;
                        }
                    } else {
                        c.begun1 = true;
                        if (++c.bar1 == Sh::kScores) c.bar1 = 0, c.turn1 ^= 1;
                    }
                    ++c.j;
                    c.t = c.j < c.end0 ? 0 : 1;
                    c.slot += 2;
                    if (c.slot == Sh::kSlots) c.slot = 0, c.phase ^= 1;
                    if (c.j >= max(c.end0, c.end1)) c.in = false, ++c.n;
                    return true;
                };
                Cursor ahead{}, at{};
                int turn_q[2] = {0, 0};
                const auto scores = [&]() {  // false: there are no more
                    if (!ahead.in && !enter(ahead)) return false;
                    if (first_of_tile(ahead))
                        ok = ok && mbar_wait_one(smem_u32(&bar_full[ahead.slot]), ahead.phase, &dead);
                    if (ahead.t == 0 ? !ahead.begun0 : !ahead.begun1) {
                        ok = ok && mbar_wait_one(smem_u32(&bar_q[ahead.t]), turn_q[ahead.t], &dead);
                        turn_q[ahead.t] ^= 1;
                    }
                    if (!ok) return false;
                    tmem_fence_after();
                    const Cursor s = ahead;
                    // over a tile of P: products are carried out in the order of their issue
                    product_columns<DP>(tmem_s(s.score), op_q + s.t * kTileStep, op_k + s.slot * kTileStep,
                                        s.j < s.narrow ? word_sinks : word_s, false);
                    mma_commit(smem_u32(&bar_s[bar_of(s)]));
                    if (s.j == (s.t == 0 ? s.end0 : s.end1) - 1) mma_commit(smem_u32(&bar_q_free[s.t]));
                    if (move(ahead)) mma_commit(smem_u32(&bar_empty[s.slot]));
                    return true;
                };
                for (int k = 0; k < Sh::kScores && scores(); ++k) {
                }
                while (ok && (at.in || enter(at))) {
                    if (first_of_tile(at))
                        ok = mbar_wait_one(smem_u32(&bar_full[at.slot + 1]), at.phase, &dead);
                    ok = ok &&
                         mbar_wait_one(smem_u32(&bar_p[bar_of(at)]), at.t == 0 ? at.turn0 : at.turn1,
                                       &dead);
                    if (!ok) break;
                    tmem_fence_after();
                    const Cursor s = at;
                    const bool add = s.t == 0 ? s.begun0 : s.begun1;
                    if (s.j < s.narrow) {
#pragma unroll
                        for (int k = 0; k < kSinkCols / 16; ++k)
                            mma_ts(tmem_o(s.t), tmem_s(s.score) + k * 8,
                                   op_v + s.slot * kTileStep + k * 128, word_o, add || k > 0);
                    } else {
                        product_rows(tmem_o(s.t), tmem_s(s.score), 32, op_v + s.slot * kTileStep, word_o,
                                     add);
                    }
                    mma_commit(smem_u32(&bar_o[bar_of(s)]));
                    scores();
                    if (move(at)) mma_commit(smem_u32(&bar_empty[s.slot + 1]));
                    if (!at.in) mbar_arrive(smem_u32(&bar_work_free[s.n % kWorks]));
                }
                mma_commit(smem_u32(&bar_drain));
                mbar_drain(smem_u32(&bar_drain), 0);
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (dead && threadIdx.x == 0) atomicAdd(p.gave_up, 1u);
    if (warp == kProductWarp) {
        __syncwarp();
        tmem_fence_after();
        tmem_free(tmem_at, 512);
    }
}

// Blocks enough for the SMs, or few of them, with their keys spread over the SMs where that saves more
// than the join costs, in units of one key tile's time.  (1,000 tokens x 8 heads x 64, 256 keys, 32
// blocks of 7 tiles: 26 us spread, 12 not; 2,000 x 8 x 128, 1,024 keys: 36 and 24.)  `window`: the keys
// that a block may walk.
constexpr int kJoin = 11;
FwdPlan plan_window(int64_t tq, int64_t tk, int batch, int heads, int64_t window) {
    const int rows = 2 * kTileRows;
    const int64_t keys = std::min((tk + kTileRows - 1) / kTileRows, window / kTileRows + 1);
    FwdPlan plan{};
    plan.whole = tiles_at_most(tq, rows, batch) * heads;
    plan.pieces = 1;
    plan.most_keys = (int)keys;
    plan.slot_rows = (int)(tq < rows ? tq : rows);
    const int64_t chunk = std::max<int64_t>(kLeastChunk, (plan.whole * keys + kSms - 1) / kSms);
    plan.spread = plan.whole < kSms && batch <= 32 && keys - chunk >= kJoin;
    return plan;
}

// Keys that a block may walk: its rows' windows, a part of a tile at either end, the sinks' tile.
int64_t walk_width(const gs_window& w) {
    return (int64_t)w.left + w.right + 1 + 2 * kTileRows + 2 * kTileRows +
           (w.sinks > 0 ? kTileRows : 0);
}

template <int DP>
cudaError_t launch_dim(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       const FwdParams& p, cudaStream_t st) {
    constexpr uint32_t kSmem = FwdShape<DP>::kSmem + kSoftmaxWarps * kStageBytes;
    static std::atomic<bool> known{false};
    cudaError_t e = launch_registers_ok(
        reinterpret_cast<const void*>(attention_window_fwd_kernel<DP>), &known);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attention_window_fwd_kernel<DP>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = p.plan.spread ? kSms : p.plan.whole;
    e = launch(attention_window_fwd_kernel<DP>, dim3((unsigned)std::min<int64_t>(blocks, kSms)),
               dim3(kWindowThreads), kSmem, st, mq, mk, mv, p, blocks);
    if (e != cudaSuccess || !p.plan.spread) return e;
    const int rows = kJoinThreads / (DP / 4);
    const unsigned y = (unsigned)((p.plan.slot_rows + rows - 1) / rows);
    return launch(attention_join_kernel<DP, true>, dim3((unsigned)p.plan.whole, y),
                  dim3(kJoinThreads), 0, st, p);
}

}  // namespace

size_t attention_window_fwd_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads,
                                            int head_dim, const gs_window& window) {
    const int64_t rows =
        plan_window(tokens_q, tokens_k, batch, heads, walk_width(window)).part_rows();
    return (size_t)rows * ((head_dim <= 64 ? 64 : 128) + 1) * sizeof(float);
}

cudaError_t launch_attention_window_fwd(const gs_attention_shape& s, const gs_window& window,
                                        const gs_heads& q, const gs_heads& k, const gs_heads& v,
                                        const gs_heads& out, float* lse, const int32_t* cu_q,
                                        const int32_t* cu_k, void* ws, cudaStream_t st) {
    FwdParams p{};
    p.batch = {cu_q, cu_k, s.tokens_q, s.tokens_k, s.batch, false};
    p.window = window_of(window, s.causal != 0);
    p.heads = s.heads_q;
    p.group = s.heads_q / s.heads_k;
    p.dim = s.head_dim;
    p.negative = s.scale < 0.f;
    // a zero scale as one too small to matter: masked scores of -infinity stay defined
    p.log2_scale = fmaxf(fabsf(s.scale) * 1.4426950408889634f, 1e-30f);
    p.o = {static_cast<__nv_bfloat16*>(out.data), out.token_stride, out.head_stride};
    p.lse = lse;
    p.plan = plan_window(s.tokens_q, s.tokens_k, s.batch, s.heads_q, walk_width(window));
    p.part_o = static_cast<float*>(ws);
    p.part_lse = p.part_o + p.plan.part_rows() * (s.head_dim <= 64 ? 64 : 128);
    CUtensorMap mq, mk, mv;
    cudaError_t e = gave_up_word(&p.gave_up);
    if (e != cudaSuccess) return e;
    e = head_map(&mq, q.data, q.token_stride, q.head_stride, s.tokens_q, s.heads_q, s.head_dim,
                 &p.swap_q);
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
