// gs_attention_window_dq.cuh -- dQ of window attention, part of gs_attention_bwd.cu: formulas, tiles
// and roundings are those of dq_block there.
//
// A block of 128 queries meets few keys (10 tiles, where 1,024 keys and 4 sinks are seen), and its
// start and end would take as long as its products.  So the CTAs go through blocks one after the
// other, as gs_attention_window_fwd.cu does: a planner takes the next block from a counter and finds
// its place, a producer brings the tiles, one thread issues the products, eight warps form dS; rings
// and barriers run on from block to block.  Which CTA takes a block does not change its result.
#pragma once

namespace gs {
namespace {

constexpr int kDqPlanner = kMathWarps + 2;
// With a window a warp more finds places and one makes the groups of four whole; registers of the
// math warps' groups and of the last one: as many in all as at launch.
constexpr int kWindowBwdThreads = kBwdThreads + 64;
constexpr int kMathRegisters = 208, kOtherRegisters = 88;
static_assert(2 * kMathRegisters + kOtherRegisters == 3 * kLaunchRegisters, "the launch's");
// Descriptions in flight: the present block's and the next one's, whose scores are formed at its end.
// The next block is taken kDqLate steps before that: earlier, a CTA keeps blocks to itself that others
// could begin (2,000 tokens x 8 heads x 128, 1,024 keys: 66 us where it took four ahead, 54 where one
// at the beginning of the one before it, 43 so).
constexpr int kDqWorks = 2, kDqLate = 5;
// who lets go of a description: the math warps, the producer and the thread of the products
constexpr int kDqReaders = kMathWarps + 2;

struct DqWork {
    Sequence sq;
    int row0, head, khead;
    int first, tiles;  // steps of the walk: those of the block's piece
    int64_t part;      // first row in the workspace (-1: the block writes the output itself)
    Walk walk;
    bool last;         // no block: the end
};

// By one whole warp: zeros for the rows of a block that sees no key.
__device__ __forceinline__ void write_no_dq(const BwdParams& p, const BwdWork& w, int dp) {
    const int lane = threadIdx.x & 31, rows = min(kTileRows, w.sq.n - w.row0);
    const bool split = w.part >= 0;
    const int words = split ? dp / 4 : p.dim / 8;  // of 16 bytes in a row
    for (int i = lane; i < rows * words; i += 32) {
        const int r = i / words, c = i - r * words;
        uint4* row = split ? reinterpret_cast<uint4*>(p.parts_q + (w.part + r) * dp)
                           : reinterpret_cast<uint4*>(p.dq.row(w.sq.q0 + w.row0 + r, w.head));
        row[c] = make_uint4(0, 0, 0, 0);
    }
}

// A CTA: its blocks of keys (gs_attention_window_dkv.cuh), then its blocks of queries.
template <int DP>
__device__ __forceinline__ void window_bwd_blocks(const CUtensorMap& map_q, const CUtensorMap& map_k,
                                                  const CUtensorMap& map_v, const CUtensorMap& map_d,
                                                  const BwdParams& p) {
    using Sh = DqShape<DP>;
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bar_q, bar_d, bar_q_free, bar_d_free, bar_s[2], bar_dp, bar_read, bar_ds[2],
        bar_dq[2], bar_raw, bar_all, bar_want;
    __shared__ uint64_t full_k[Sh::kSlotsK], empty_k[Sh::kSlotsK], full_v[Sh::kSlotsV],
        empty_v[Sh::kSlotsV], bar_work[kDqWorks], bar_work_free[kDqWorks];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    __shared__ DqWork works[kDqWorks];
    __shared__ DkvState<DP> dkv;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t at_q = smem, at_d = smem + Sh::kTileBytes;
    const uint32_t at_k = smem + 2 * Sh::kTileBytes, at_v = at_k + Sh::kSlotsK * Sh::kTileBytes;
    if (warp == kMathWarps) {
        tmem_alloc(smem_u32(&tmem_at), 512);
    } else if (threadIdx.x == 0) {
        dead = 0;
        for (uint64_t* b : {&bar_q, &bar_d, &bar_q_free, &bar_d_free, &bar_s[0], &bar_s[1], &bar_dp,
                            &bar_dq[0], &bar_dq[1], &bar_raw, &bar_all, &bar_want})
            mbar_init(smem_u32(b), 1);
        for (uint64_t* b : {&bar_ds[0], &bar_ds[1], &bar_read}) mbar_init(smem_u32(b), kMathWarps);
        for (int i = 0; i < Sh::kSlotsK; ++i) {
            mbar_init(smem_u32(&full_k[i]), 1);
            mbar_init(smem_u32(&empty_k[i]), 1);
        }
        for (int i = 0; i < Sh::kSlotsV; ++i) {
            mbar_init(smem_u32(&full_v[i]), 1);
            mbar_init(smem_u32(&empty_v[i]), 1);
        }
        for (int i = 0; i < kDqWorks; ++i) {
            mbar_init(smem_u32(&bar_work[i]), 1);
            mbar_init(smem_u32(&bar_work_free[i]), kDqReaders);
        }
        dkv.init();
        fence_barrier_init();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // all 512 columns are the CTA's: their addresses start at 0
    constexpr uint32_t tmem = 0, t_dp = 256, t_dq = 384;
    // Between the two kinds of blocks: all warps are through with the first, whose shared and tensor
    // memory the second one takes.  False: a wait has given up.
    const auto next_kind = [&]() {
        tmem_fence_before();
        fence_async_shared();
        __syncthreads();
        tmem_fence_after();
        return !any_dead(&dead);
    };

    if (warp < kMathWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMathRegisters));
        dkv_math<DP>(p, smem_raw, smem, dkv, &dead);
        bool go = next_kind();
        // ---- dS: one query a thread, half of the tile's keys ----
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t dp_at = t_dp + lanes + half * 64;
        const float sl = p.log2_scale;
        const float2 sl2 = make_float2(sl, sl);
        int x = 0;  // steps of all blocks
        for (int n = 0; go; ++n) {
            const int slot = n % kDqWorks;
            if (!mbar_wait(smem_u32(&bar_work[slot]), (n / kDqWorks) & 1, &dead)) break;
            const DqWork& w = works[slot];
            if (w.last) break;
            const int row = w.row0 + r, tiles = w.tiles;
            // the first key of step j in the warps' half: behind the sinks' tile one follows another
            const int key0 = (w.walk.first + w.first - w.walk.extra) * kTileRows + half * 64;
            const int sink_steps = w.walk.extra - w.first;
            float nl = -INFINITY, nd = 0.f;
            if (row < w.sq.n) {
                const int64_t at = (int64_t)w.head * p.batch.tq + w.sq.q0 + row;
                nl = p.nlse[at];
                nd = p.ndelta[at];
            }
            // what the row sees, the end of the warp's first row's keys and the start of its last
            // one's
            const Seen see = seen_by(p.window, row, w.sq.n, w.sq.m);
            const int first_hi = __shfl_sync(0xffffffffu, see.hi, 0);
            const int last_lo = __shfl_sync(0xffffffffu, see.lo, 31);
            const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
            for (int j = 0; j < tiles; ++j, ++x) {
                const uint32_t s_at = tmem + (x & 1) * 128 + lanes + half * 64;
                mbar_pass(smem_u32(&bar_s[x & 1]), (x >> 1) & 1, &dead);
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
                mbar_pass(smem_u32(&bar_dp), x & 1, &dead);
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
                const int key = j < sink_steps ? half * 64 : key0 + j * kTileRows;
                if (key + 64 > first_hi || key < last_lo) {
#pragma unroll
                    for (int c = 0; c < 64; c += 32)
                        mask_by_bits(dp + c,
                                     seen_bits(see.lo - key - c, see.hi - key - c,
                                               see.sinks - key - c),
                                     0.f);
                }
                store_half(s_at, dp);
                tmem_wait_st();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_ds[x & 1]));
            }
            mbar_pass(smem_u32(&bar_dq[n & 1]), (n >> 1) & 1, &dead);
            if (any_dead(&dead)) break;
            tmem_fence_after();
            // each half of the warps writes half of the columns
            const int c0 = half * (DP / 2), rows = w.sq.n - (row - lane);
            __nv_bfloat16* out = p.dq.row(w.sq.q0 + row - lane, w.head) + c0;
            float* part = w.part >= 0 ? p.parts_q + (w.part + r - lane) * DP + c0 : nullptr;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_work_free[slot]));
            store_rows<DP / 2, DP>(t_dq + lanes + c0, out, p.dq.ts, part, 0, rows, p.dim - c0, p.scale,
                                   false);
            tmem_fence_before();  // dQ may be written over once the next dS is there
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegisters));
        if (warp == kDqPlanner) {
            // ---- the planner ----
            dkv_plan<DP>(p, dkv, &dead);
            const bool go = next_kind();
            const int64_t blocks = blocks_of(p.plan_q);
            int n = 0;  // descriptions so far
            bool taken = false;  // whether block n has been asked for
            while (go) {
                if (n > 0 && !taken && !mbar_wait_block(smem_u32(&bar_want), (n - 1) & 1, &dead)) break;
                taken = true;
                unsigned int next = 0;
                if (lane == 0) next = atomicAdd(p.next_dq, 1u);
                const int64_t id = __shfl_sync(0xffffffffu, next, 0);
                const bool end = id >= blocks;
                __shared__ BwdWork found;
                if (!end) {
                    if (!find_work<false, true>(p, id, &found)) continue;
                    __syncwarp();
                    if (found.items == 0) {
                        write_no_dq(p, found, DP);
                        __syncwarp();
                        continue;
                    }
                }
                const int slot = n % kDqWorks, use = n / kDqWorks;
                if (use > 0 && !mbar_wait_block(smem_u32(&bar_work_free[slot]), (use - 1) & 1, &dead))
                    break;
                if (lane == 0) {
                    DqWork& w = works[slot];
                    w.last = end;
                    if (!end) {
                        w.sq = found.sq;
                        w.row0 = found.row0;
                        w.head = found.head;
                        w.khead = found.khead;
                        w.first = found.first;
                        w.tiles = found.items;
                        w.part = found.part;
                        w.walk = found.walk;
                    }
                    mbar_arrive(smem_u32(&bar_work[slot]));
                }
                __syncwarp();
                ++n;
                taken = false;
                if (end) break;
            }
        } else if (warp == kMathWarps + 1) {
            // ---- the producer: Q, the first K, dO, then V and K in turn ----
            dkv_bring<DP>(map_q, map_k, map_v, map_d, p, smem_raw, smem, dkv, &dead);
            int blocks = 0, tiles_k = 0, tiles_v = 0, mends = 0;  // brought so far
            int loads_q = 0, loads_d = 0;
            bool ok = next_kind();
            for (; ok; ++blocks) {
                const int at = blocks % kDqWorks;
                if (!mbar_wait_block(smem_u32(&bar_work[at]), (blocks / kDqWorks) & 1, &dead)) break;
                if (works[at].last) break;
                const DqWork w = works[at];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_work_free[at]));
                const int64_t q = w.sq.q0 + w.row0;
                const bool tail = w.sq.k0 + w.sq.m < p.batch.tk;
                if (loads_q > 0) ok = mbar_wait(smem_u32(&bar_q_free), (loads_q - 1) & 1, &dead);
                if (!ok) break;
                if (elect_one()) {
                    mbar_expect(smem_u32(&bar_q), Sh::kTileBytes);
                    load_tile<Sh::kBlocks>(at_q, &map_q, smem_u32(&bar_q), w.head, q, p.swap_q);
                }
                __syncwarp();
                ++loads_q;
                for (int j = 0; j < w.tiles; ++j) {
                    const int tile = w.walk.tile(w.first + j);
                    const int64_t token = w.sq.k0 + (int64_t)tile * kTileRows;
                    const int sk = tiles_k % Sh::kSlotsK, uk = tiles_k / Sh::kSlotsK;
                    const int sv = tiles_v % Sh::kSlotsV, uv = tiles_v / Sh::kSlotsV;
                    if (uk > 0) ok = mbar_wait(smem_u32(&empty_k[sk]), (uk - 1) & 1, &dead);
                    if (!ok) break;
                    // keys of another sequence behind this one's end: zeros in their place
                    const int valid = w.sq.m - tile * kTileRows;
                    const bool mend = valid < kTileRows && tail;
                    const uint32_t full = smem_u32(&full_k[sk]), dst = at_k + sk * Sh::kTileBytes;
                    const uint32_t bar = mend ? smem_u32(&bar_raw) : full;
                    if (elect_one()) {
                        mbar_expect(bar, Sh::kTileBytes);
                        load_tile<Sh::kBlocks>(dst, &map_k, bar, w.khead, token, p.swap_k);
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
                        __syncwarp();
                    }
                    ++tiles_k;
                    if (j == 0) {
                        if (loads_d > 0) ok = mbar_wait(smem_u32(&bar_d_free), (loads_d - 1) & 1, &dead);
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_expect(smem_u32(&bar_d), Sh::kTileBytes);
                            load_tile<Sh::kBlocks>(at_d, &map_d, smem_u32(&bar_d), w.head, q, p.swap_d);
                        }
                        __syncwarp();
                        ++loads_d;
                    }
                    if (uv > 0) ok = mbar_wait(smem_u32(&empty_v[sv]), (uv - 1) & 1, &dead);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_expect(smem_u32(&full_v[sv]), Sh::kTileBytes);
                        load_tile<Sh::kBlocks>(at_v + sv * Sh::kTileBytes, &map_v,
                                               smem_u32(&full_v[sv]), w.khead, token, p.swap_v);
                    }
                    ++tiles_v;
                    __syncwarp();
                }
            }
            if (loads_q > 0) mbar_drain(smem_u32(&bar_q), (loads_q - 1) & 1);
            if (loads_d > 0) mbar_drain(smem_u32(&bar_d), (loads_d - 1) & 1);
            drain_ring<Sh::kSlotsK>(full_k, tiles_k);
            drain_ring<Sh::kSlotsV>(full_v, tiles_v);
        } else if (warp == kMathWarps) {
            // ---- the products ----
            if (elect_one()) dkv_multiply<DP>(p, smem_raw, smem, dkv, &dead);
            __syncwarp();
            if (next_kind() && elect_one()) {
                constexpr uint32_t word_o = mma_word(128, DP, false, true);
                constexpr uint32_t word_dp = mma_word(128, 128, false, false);
                const uint32_t word_s = word_dp | (p.negative ? kNegateA : 0u);
                bool ok = true;
                // places in the rings, which run on through the blocks: K of the scores and of dQ, V
                int k_s = 0, k_s_phase = 0, k_q = 0, v = 0, v_phase = 0;
                // steps so far of the scores, of dO V^T, of dQ (their parities are what counts)
                int of_s = 0, of_p = 0, of_q = 0;
                int blocks_s = 0, blocks_p = 0;  // that have begun
                const auto scores = [&](bool first, bool last) {
                    ok = ok && mbar_wait_one(smem_u32(&full_k[k_s]), k_s_phase, &dead);
                    if (first) ok = ok && mbar_wait_one(smem_u32(&bar_q), blocks_s++ & 1, &dead);
                    if (!ok) return;
                    tmem_fence_after();
                    product_columns<DP>(tmem + (of_s & 1) * 128, operand_columns(at_q),
                                        operand_columns(at_k + k_s * Sh::kTileBytes), word_s, false);
                    mma_commit(smem_u32(&bar_s[of_s & 1]));
                    if (last) mma_commit(smem_u32(&bar_q_free));
                    ++of_s;
                    if (++k_s == Sh::kSlotsK) k_s = 0, k_s_phase ^= 1;
                };
                const auto dprobs = [&](bool first, bool last) {
                    // once the one before is read
                    if (of_p > 0) ok = ok && mbar_wait_one(smem_u32(&bar_read), (of_p - 1) & 1, &dead);
                    ok = ok && mbar_wait_one(smem_u32(&full_v[v]), v_phase, &dead);
                    if (first) ok = ok && mbar_wait_one(smem_u32(&bar_d), blocks_p++ & 1, &dead);
                    if (!ok) return;
                    tmem_fence_after();
                    product_columns<DP>(t_dp, operand_columns(at_d),
                                        operand_columns(at_v + v * Sh::kTileBytes), word_dp, false);
                    mma_commit(smem_u32(&bar_dp));
                    mma_commit(smem_u32(&empty_v[v]));
                    if (last) mma_commit(smem_u32(&bar_d_free));
                    ++of_p;
                    if (++v == Sh::kSlotsV) v = 0, v_phase ^= 1;
                };
                // the steps of block n, or 0 behind the last one
                const auto steps_of = [&](int n) {
                    const int i = n % kDqWorks;
                    ok = ok && mbar_wait_one(smem_u32(&bar_work[i]), (n / kDqWorks) & 1, &dead);
                    return !ok || works[i].last ? 0 : works[i].tiles;
                };
                int tiles = steps_of(0);
                for (int n = 0; tiles > 0; ++n) {
                    // scores run two steps ahead of dQ, dO V^T one: those of another block's first
                    // steps come from the end of the block before it
                    if (n == 0) {
                        scores(true, tiles == 1);
                        dprobs(true, tiles == 1);
                        if (tiles > 1) scores(false, tiles == 2);
                    }
                    int next = -1;
                    for (int j = 0; j < tiles && ok; ++j) {
                        if (j == max(0, tiles - kDqLate)) mbar_arrive(smem_u32(&bar_want));
                        // the next dO V^T as soon as this one is read, while dS is formed from it
                        if (j + 1 < tiles) dprobs(false, j + 2 == tiles);
                        ok = ok && mbar_wait_one(smem_u32(&bar_ds[of_q & 1]), (of_q >> 1) & 1, &dead);
                        if (!ok) break;
                        tmem_fence_after();
                        product_rows(t_dq, tmem + (of_q & 1) * 128, 64,
                                     operand_rows(at_k + k_q * Sh::kTileBytes), word_o, j > 0);
                        mma_commit(smem_u32(&empty_k[k_q]));
                        ++of_q;
                        if (++k_q == Sh::kSlotsK) k_q = 0;
                        if (j + 2 < tiles) {
                            scores(false, j + 3 == tiles);
                        } else if (next < 0) {
                            if (j + 1 == tiles) mma_commit(smem_u32(&bar_dq[n & 1]));
                            next = steps_of(n + 1);
                            if (next > 0) scores(true, next == 1);
                        }
                    }
                    if (!ok) break;
                    if (tiles > 1) mma_commit(smem_u32(&bar_dq[n & 1]));
                    mbar_arrive(smem_u32(&bar_work_free[n % kDqWorks]));
                    if (next > 0) dprobs(true, next == 1);
                    if (next > 1) scores(false, next == 2);
                    tiles = next;
                }
                mma_commit(smem_u32(&bar_all));
                mbar_drain(smem_u32(&bar_all), 0);
            }
        } else {
            next_kind();
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

}  // namespace
}  // namespace gs
