// gs_attention_window_dkv.cuh -- dK and dV of window attention, part of gs_attention_bwd.cu: formulas,
// tiles and roundings are those of dkv_block there.
//
// As the blocks of queries (gs_attention_window_dq.cuh) a CTA goes through blocks of keys one after the
// other: while a block's dK and dV are on their way to memory the next one's tiles arrive and its first
// products are formed.  The blocks of the sinks come first, since every query may see them.  Here are
// the roles' parts, which the CTA's warps go through before those of the blocks of queries.
#pragma once

namespace gs {
namespace {

// Descriptions in flight, and how many steps before a block's end the next one is taken: see kDqWorks.
// (2,500 + 1,104 tokens x 8 heads x 64, 513 keys: 41.9 us with 2, 41.0 with 4, 41.3 with 8; a CTA a block
// 44.9.)
constexpr int kDkvWorks = 2, kDkvLate = 4;
// who lets go of a description: the math warps, the producer and the thread of the products
constexpr int kDkvReaders = kMathWarps + 2;

struct DkvWork {
    Sequence sq;
    int row0, khead;
    int first, items;        // query tiles of all heads that share the keys: those of the block's piece
    int q_first, per_head;   // query tiles of a head
    int key_first, key_end;  // keys that the block writes, less row0
    int64_t part;            // first row in the workspace (-1: the block writes the outputs itself)
    bool sinks, last;        // a block of the sinks; no block: the end
};

template <int DP>
struct DkvState {
    using Sh = DkvShape<DP>;
    uint64_t bar_k, bar_v, bar_k_free, bar_v_free, bar_s, bar_dp[Sh::kDp], bar_p, bar_ds[Sh::kDp],
        bar_done, bar_out_free, bar_raw, bar_all, bar_want, bar_kept, bar_join;
    uint64_t full_q[Sh::kSlots], empty_q[Sh::kSlots], full_d[Sh::kSlots], empty_d[Sh::kSlots],
        bar_work[kDkvWorks], bar_work_free[kDkvWorks];
    DkvWork works[kDkvWorks];
    BwdWork found;
    int join;  // whether the block's sinks are to be joined

    __device__ __forceinline__ void init() {
        for (uint64_t* b : {&bar_k, &bar_v, &bar_k_free, &bar_v_free, &bar_s, &bar_done, &bar_raw,
                            &bar_all, &bar_want, &bar_join})
            mbar_init(smem_u32(b), 1);
        for (uint64_t* b : {&bar_p, &bar_out_free, &bar_kept}) mbar_init(smem_u32(b), kMathWarps);
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
        for (int i = 0; i < kDkvWorks; ++i) {
            mbar_init(smem_u32(&bar_work[i]), 1);
            mbar_init(smem_u32(&bar_work_free[i]), kDkvReaders);
        }
    }
};

// where the tiles, and -lse log2(e) and -delta of each slot's queries, lie in shared memory
template <int DP>
struct DkvPlaces {
    using Sh = DkvShape<DP>;
    uint32_t k, v, q, d;
    float (*rows)[2][kTileRows];
    __device__ __forceinline__ DkvPlaces(char* raw, uint32_t smem) {
        k = smem;
        v = k + Sh::kTileBytes;
        q = v + Sh::kTileBytes;
        d = q + Sh::kSlots * Sh::kTileBytes;
        rows = reinterpret_cast<float(*)[2][kTileRows]>(raw + (smem + Sh::kRows - smem_u32(raw)));
    }
};

// The sums of a block of keys as rows in the workspace: dK, and dV behind it.
template <int DP>
__device__ __forceinline__ float* dkv_parts(const BwdParams& p, bool sinks, int64_t part, bool of_v) {
    return sinks ? p.parts_s + (part + (of_v ? p.window.sinks : 0)) * DP
                 : p.parts_k + (part + (of_v ? part_rows(p.plan_k) : 0)) * DP;
}

// By one whole warp: zeros for the keys of a block that no query sees.
template <int DP>
__device__ __forceinline__ void write_no_dkv(const BwdParams& p, const BwdWork& w) {
    const int lane = threadIdx.x & 31, rows = w.key_end - w.key_first;
    const bool split = w.part >= 0;
    const int words = split ? DP / 4 : p.dim / 8;  // of 16 bytes in a row
    for (int of_v = 0; of_v < 2; ++of_v) {
        const HeadView& g = of_v ? p.dv : p.dk;
        for (int i = lane; i < rows * words; i += 32) {
            const int r = i / words + w.key_first, c = i % words;
            uint4* row =
                split ? reinterpret_cast<uint4*>(dkv_parts<DP>(p, false, w.part + r, of_v))
                      : reinterpret_cast<uint4*>(g.row(w.sq.k0 + w.row0 + r, w.khead));
            row[c] = make_uint4(0, 0, 0, 0);
        }
    }
}

// dK and dV of the sinks of a sequence that several blocks took, in the blocks' order, by the math
// warps of the one that is done last.  DP / 4 lanes a row.  (By a kernel behind this one: 4 us more.)
// The warps meet at barriers whose waits are bounded, as all here: some of them may have left where a
// wait gave up, and at a barrier of the hardware the others would stay for ever.  `joins`: such blocks
// of this CTA before this one.  False: a wait has given up.
template <int DP>
__device__ __forceinline__ bool join_sinks(const BwdParams& p, const DkvWork& w, DkvState<DP>& sh,
                                           int joins, volatile int* dead) {
    const Sequence sq = w.sq;
    const int64_t slot = sink_slot(sq.q0, p.sink_rows);
    const int pieces = (sq.n + p.sink_rows - 1) / p.sink_rows, sinks = p.window.sinks;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sh.bar_kept));  // the warp's rows are kept
    if (threadIdx.x < 32) {
        if (!mbar_wait(smem_u32(&sh.bar_kept), joins & 1, dead)) return false;
        if (threadIdx.x == 0) {
            __threadfence();
            sh.join =
                atomicAdd(p.sinks_done + slot * p.heads_k + w.khead, 1u) == (unsigned)pieces - 1;
            __threadfence();
            mbar_arrive(smem_u32(&sh.bar_join));
        }
        __syncwarp();
    }
    if (!mbar_wait(smem_u32(&sh.bar_join), joins & 1, dead)) return false;
    if (!sh.join) return true;
    constexpr int kLanes = DP / 4;
    const int lane = threadIdx.x % kLanes;
    for (int r = threadIdx.x / kLanes; r < 2 * w.key_end; r += kMathWarps * 32 / kLanes) {
        const bool of_v = r >= w.key_end;
        const int key = of_v ? r - w.key_end : r;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int z = 0; z < pieces; ++z) {
            const int64_t row = ((slot + z) * p.heads_k + w.khead) * 2 * sinks + (of_v ? sinks : 0) + key;
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.parts_s) + row * kLanes + lane);
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
        }
        const float f = of_v ? 1.f : p.scale;
        if (lane * 4 < p.dim)
            *reinterpret_cast<uint2*>((of_v ? p.dv : p.dk).row(sq.k0 + key, w.khead) + lane * 4) =
                make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
    }
    return true;
}

// ---- the planner: one whole warp ----
template <int DP>
__device__ __forceinline__ void dkv_plan(const BwdParams& p, DkvState<DP>& sh, volatile int* dead) {
    const int lane = threadIdx.x & 31;
    const int64_t blocks = p.sink_blocks + blocks_of(p.plan_k);
    int n = 0;  // descriptions so far
    bool taken = false;  // whether block n has been asked for
    for (;;) {
        if (n > 0 && !taken && !mbar_wait_block(smem_u32(&sh.bar_want), (n - 1) & 1, dead)) break;
        taken = true;
        unsigned int next = 0;
        if (lane == 0) next = atomicAdd(p.next_dkv, 1u);
        const int64_t id = __shfl_sync(0xffffffffu, next, 0);
        const bool end = id >= blocks, sinks = id < p.sink_blocks;
        if (!end) {
            const bool there = sinks ? find_sink_work(p, id, &sh.found)
                                     : find_work<true, true>(p, id - p.sink_blocks, &sh.found);
            if (!there) continue;
            __syncwarp();
            if (sh.found.items == 0) {
                write_no_dkv<DP>(p, sh.found);
                __syncwarp();
                continue;
            }
        }
        const int slot = n % kDkvWorks, use = n / kDkvWorks;
        if (use > 0 && !mbar_wait_block(smem_u32(&sh.bar_work_free[slot]), (use - 1) & 1, dead)) break;
        if (lane == 0) {
            DkvWork& w = sh.works[slot];
            w.last = end;
            if (!end) {
                const BwdWork& f = sh.found;
                w.sq = f.sq;
                w.row0 = f.row0;
                w.khead = f.khead;
                w.first = f.first;
                w.items = f.items;
                w.q_first = f.q_first;
                w.per_head = f.per_head;
                w.key_first = f.key_first;
                w.key_end = f.key_end;
                w.part = f.part;
                w.sinks = sinks;
            }
            mbar_arrive(smem_u32(&sh.bar_work[slot]));
        }
        __syncwarp();
        ++n;
        taken = false;
        if (end) break;
    }
}

// ---- the producer, one whole warp: K, the first Q, V, then dO and Q in turn ----
template <int DP>
__device__ __forceinline__ void dkv_bring(const CUtensorMap& map_q, const CUtensorMap& map_k,
                                          const CUtensorMap& map_v, const CUtensorMap& map_d,
                                          const BwdParams& p, char* raw, uint32_t smem,
                                          DkvState<DP>& sh, volatile int* dead) {
    using Sh = DkvShape<DP>;
    const int lane = threadIdx.x & 31;
    const DkvPlaces<DP> at(raw, smem);
    uint64_t *full_q = sh.full_q, *full_d = sh.full_d;
    int loads_k = 0, loads_v = 0, tiles_q = 0, tiles_d = 0, mends = 0;  // brought so far
    bool ok = true;
    for (int n = 0; ok; ++n) {
        const int slot_w = n % kDkvWorks;
        if (!mbar_wait_block(smem_u32(&sh.bar_work[slot_w]), (n / kDkvWorks) & 1, dead)) break;
        if (sh.works[slot_w].last) break;
        const DkvWork w = sh.works[slot_w];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.bar_work_free[slot_w]));
        const Sequence sq = w.sq;
        const int64_t key = sq.k0 + w.row0;
        // one tile of queries or (of_d) of output gradients
        const auto bring = [&](bool of_d, uint32_t dst, uint32_t full, int head, int i0) {
            const int valid = sq.n - i0;
            // rows of another sequence behind this one's end: zeros in their place
            const bool mend = valid < kTileRows && sq.q0 + sq.n < p.batch.tq;
            const uint32_t bar = mend ? smem_u32(&sh.bar_raw) : full;
            if (elect_one()) {
                mbar_expect(bar, Sh::kTileBytes);
                load_tile<Sh::kBlocks>(dst, of_d ? &map_d : &map_q, bar, head, sq.q0 + i0,
                                       of_d ? p.swap_d : p.swap_q);
            }
            __syncwarp();
            if (mend) {
                const int parity = mends++ & 1;
                ok = mbar_wait(bar, parity, dead);
                if (!ok) {
                    mbar_drain(bar, parity);
                    return;
                }
                zero_rows<Sh::kBlocks>(raw + (dst - smem_u32(raw)), valid);
                fence_async_shared();
                __syncwarp();
                if (elect_one()) mbar_arrive(full);
                __syncwarp();
            }
        };
        // K or V, once the last block's products with it are done
        const auto bring_keys = [&](const CUtensorMap& map, uint64_t* bar, uint64_t* bar_free, uint32_t dst,
                                    bool swap, int& loads) {
            if (loads > 0) ok = mbar_wait(smem_u32(bar_free), (loads - 1) & 1, dead);
            if (!ok) return;
            if (elect_one()) {
                mbar_expect(smem_u32(bar), Sh::kTileBytes);
                load_tile<Sh::kBlocks>(dst, &map, smem_u32(bar), w.khead, key, swap);
            }
            __syncwarp();
            ++loads;
        };
        bring_keys(map_k, &sh.bar_k, &sh.bar_k_free, at.k, p.swap_k, loads_k);
        if (!ok) break;
        int head = w.khead * p.group + w.first / w.per_head, tile = w.q_first + w.first % w.per_head;
        for (int i = 0; i < w.items; ++i) {
            const int slot = tiles_q % Sh::kSlots, use = tiles_q / Sh::kSlots, i0 = tile * kTileRows;
            if (use > 0) ok = mbar_wait(smem_u32(&sh.empty_q[slot]), (use - 1) & 1, dead);
            if (!ok) break;
            const uint32_t full = smem_u32(&full_q[slot]);
            bring(false, at.q + slot * Sh::kTileBytes, full, head, i0);
            if (!ok) break;
            const int64_t src = (int64_t)head * p.batch.tq + sq.q0 + i0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = k * 32 + lane;
                at.rows[slot][0][r] = i0 + r < sq.n ? p.nlse[src + r] : -INFINITY;
                at.rows[slot][1][r] = i0 + r < sq.n ? p.ndelta[src + r] : 0.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
            ++tiles_q;
            if (i == 0) bring_keys(map_v, &sh.bar_v, &sh.bar_v_free, at.v, p.swap_v, loads_v);
            if (!ok) break;
            if (use > 0) ok = mbar_wait(smem_u32(&sh.empty_d[slot]), (use - 1) & 1, dead);
            if (!ok) break;
            bring(true, at.d + slot * Sh::kTileBytes, smem_u32(&full_d[slot]), head, i0);
            if (!ok) break;
            ++tiles_d;
            if (++tile == w.q_first + w.per_head) tile = w.q_first, ++head;
        }
    }
    if (loads_k > 0) mbar_drain(smem_u32(&sh.bar_k), (loads_k - 1) & 1);
    if (loads_v > 0) mbar_drain(smem_u32(&sh.bar_v), (loads_v - 1) & 1);
    drain_ring<Sh::kSlots>(full_q, tiles_q);
    drain_ring<Sh::kSlots>(full_d, tiles_d);
}

// tensor memory: S, dO V^T (with two of them the next one is formed before dS of this one is), dV, dK
template <int DP>
struct DkvColumns {
    static constexpr uint32_t s = 0, dp = 128, dv = dp + DkvShape<DP>::kDp * 128, dk = dv + DP;
};

// ---- the products: one thread ----
template <int DP>
__device__ __forceinline__ void dkv_multiply(const BwdParams& p, char* raw, uint32_t smem,
                                             DkvState<DP>& sh, volatile int* dead) {
    using Sh = DkvShape<DP>;
    using At = DkvColumns<DP>;
    const DkvPlaces<DP> at(raw, smem);
    constexpr uint32_t word_o = mma_word(128, DP, false, true);
    constexpr uint32_t word_dp = mma_word(128, 128, false, false);
    const uint32_t word_s = word_dp | (p.negative ? kNegateA : 0u);
    bool ok = true;
    int of_s = 0, of_p = 0, x = 0;   // steps so far of the scores, of dO V^T, of all products
    int blocks_s = 0, blocks_p = 0;  // that have begun
    const auto scores = [&](bool first, bool last) {
        const int slot = of_s % Sh::kSlots;
        ok = ok && mbar_wait_one(smem_u32(&sh.full_q[slot]), (of_s / Sh::kSlots) & 1, dead);
        if (first) ok = ok && mbar_wait_one(smem_u32(&sh.bar_k), blocks_s++ & 1, dead);
        if (!ok) return;
        tmem_fence_after();
        product_columns<DP>(At::s, operand_columns(at.k), operand_columns(at.q + slot * Sh::kTileBytes),
                            word_s, false);
        mma_commit(smem_u32(&sh.bar_s));
        if (last) mma_commit(smem_u32(&sh.bar_k_free));
        ++of_s;
    };
    const auto dprobs = [&](bool first, bool last) {
        const int slot = of_p % Sh::kSlots;
        ok = ok && mbar_wait_one(smem_u32(&sh.full_d[slot]), (of_p / Sh::kSlots) & 1, dead);
        if (first) ok = ok && mbar_wait_one(smem_u32(&sh.bar_v), blocks_p++ & 1, dead);
        if (!ok) return;
        tmem_fence_after();
        product_columns<DP>(At::dp + of_p % Sh::kDp * 128, operand_columns(at.v),
                            operand_columns(at.d + slot * Sh::kTileBytes), word_dp, false);
        mma_commit(smem_u32(&sh.bar_dp[of_p % Sh::kDp]));
        if (last) mma_commit(smem_u32(&sh.bar_v_free));
        ++of_p;
    };
    // the steps of block n, or 0 behind the last one
    const auto steps_of = [&](int n) {
        const int i = n % kDkvWorks;
        ok = ok && mbar_wait_one(smem_u32(&sh.bar_work[i]), (n / kDkvWorks) & 1, dead);
        return !ok || sh.works[i].last ? 0 : sh.works[i].items;
    };
    int items = steps_of(0);
    for (int n = 0; items > 0; ++n) {
        // (a block behind the first: while the last one's results are on their way to memory)
        scores(true, items == 1);
        dprobs(true, items == 1);
        for (int i = 0; i < items && ok; ++i, ++x) {
            if (i == max(0, items - kDkvLate)) mbar_arrive(smem_u32(&sh.bar_want));
            const int slot = x % Sh::kSlots;
            // while the other warps form dS: dV, and the next scores
            ok = mbar_wait_one(smem_u32(&sh.bar_p), x & 1, dead);
            if (i == 0 && n > 0)  // the last block's results are read
                ok = ok && mbar_wait_one(smem_u32(&sh.bar_out_free), (n - 1) & 1, dead);
            if (!ok) break;
            tmem_fence_after();
            product_rows(At::dv, At::s, 64, operand_rows(at.d + slot * Sh::kTileBytes), word_o, i > 0);
            mma_commit(smem_u32(&sh.empty_d[slot]));
            if (i + 1 < items) scores(false, i + 2 == items);
            if (Sh::kDp == 2 && i + 1 < items) dprobs(false, i + 2 == items);
            // while they form the next P: dK, and the next dO V^T
            ok = ok && mbar_wait_one(smem_u32(&sh.bar_ds[x % Sh::kDp]), (x / Sh::kDp) & 1, dead);
            if (!ok) break;
            tmem_fence_after();
            product_rows(At::dk, At::dp + x % Sh::kDp * 128, 64,
                         operand_rows(at.q + slot * Sh::kTileBytes), word_o, i > 0);
            mma_commit(smem_u32(&sh.empty_q[slot]));
            if (Sh::kDp == 1 && i + 1 < items) dprobs(false, i + 2 == items);
        }
        if (!ok) break;
        mma_commit(smem_u32(&sh.bar_done));
        mbar_arrive(smem_u32(&sh.bar_work_free[n % kDkvWorks]));
        items = steps_of(n + 1);
    }
    mma_commit(smem_u32(&sh.bar_all));
    mbar_drain(smem_u32(&sh.bar_all), 0);
}

// ---- P and dS, the math warps: one key a thread, half of the tile's queries ----
template <int DP>
__device__ __forceinline__ void dkv_math(const BwdParams& p, char* raw, uint32_t smem,
                                         DkvState<DP>& sh, volatile int* dead) {
    using Sh = DkvShape<DP>;
    using At = DkvColumns<DP>;
    const DkvPlaces<DP> at(raw, smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = At::s + lanes + half * 64;
    const float2 sl2 = make_float2(p.log2_scale, p.log2_scale);
    int x = 0;      // steps of all blocks
    int joins = 0;  // blocks so far whose sinks' sums are kept
    for (int n = 0;; ++n) {
        const int slot_w = n % kDkvWorks;
        if (!mbar_wait(smem_u32(&sh.bar_work[slot_w]), (n / kDkvWorks) & 1, dead)) break;
        const DkvWork& w = sh.works[slot_w];
        if (w.last) break;
        const int items = w.items, q_first = w.q_first, q_end = w.q_first + w.per_head;
        // the queries that see this thread's key; of the tile's keys the last first one, the first
        // behind the last
        int sees, sees_end, all_see, all_end, unused;
        seers_of(p.window, w.row0 + r, w.sq.n, w.sq.m, &sees, &sees_end);
        seers_of(p.window, w.row0 + w.key_first, w.sq.n, w.sq.m, &unused, &all_end);
        seers_of(p.window, w.row0 + w.key_end - 1, w.sq.n, w.sq.m, &all_see, &unused);
        int tile = q_first + w.first % w.per_head;
        for (int i = 0; i < items; ++i, ++x) {
            const int slot = x % Sh::kSlots, i0 = tile * kTileRows;
            if (++tile == q_end) tile = q_first;
            const bool masked = i0 < all_see || i0 + kTileRows > all_end;
            const int lo = sees - i0 - half * 64, hi = sees_end - i0 - half * 64;
            mbar_pass(smem_u32(&sh.full_q[slot]), (x / Sh::kSlots) & 1, dead);
            mbar_pass(smem_u32(&sh.bar_s), x & 1, dead);
            tmem_fence_after();
            float pr[64];
            tmem_ld32(reinterpret_cast<uint32_t*>(pr), s_at);
            tmem_ld32(reinterpret_cast<uint32_t*>(pr) + 32, s_at + 32);
            tmem_wait_ld();
            const float4* nl = reinterpret_cast<const float4*>(at.rows[slot][0] + half * 64);
            const float4* nd = reinterpret_cast<const float4*>(at.rows[slot][1] + half * 64);
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
                mask_by_bits(pr, seen_bits(lo, hi, 0), 0.f);
                mask_by_bits(pr + 32, seen_bits(lo - 32, hi - 32, 0), 0.f);
            }
            store_half(s_at, pr);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.bar_p));
            const uint32_t dp_at = At::dp + x % Sh::kDp * 128 + lanes + half * 64;
            mbar_pass(smem_u32(&sh.bar_dp[x % Sh::kDp]), (x / Sh::kDp) & 1, dead);
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
                mask_by_bits(dp, seen_bits(lo, hi, 0), 0.f);
                mask_by_bits(dp + 32, seen_bits(lo - 32, hi - 32, 0), 0.f);
            }
            store_half(dp_at, dp);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.bar_ds[x % Sh::kDp]));
        }
        mbar_pass(smem_u32(&sh.bar_done), n & 1, dead);
        if (any_dead(dead)) break;
        tmem_fence_after();
        // half of the warps write dV, half dK
        const int row = (warp & 3) * 32;  // the warp's first
        const HeadView& g = half ? p.dk : p.dv;
        const bool split = w.part >= 0;
        store_rows<DP, DP>((half ? At::dk : At::dv) + lanes, g.row(w.sq.k0 + w.row0 + row, w.khead), g.ts,
                           split ? dkv_parts<DP>(p, w.sinks, w.part + row, !half) : nullptr,
                           w.key_first - row, w.key_end - row, p.dim, half ? p.scale : 1.f, false);
        tmem_fence_before();  // they may be written over
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.bar_out_free));
        if (w.sinks && split && !join_sinks<DP>(p, w, sh, joins++, dead)) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.bar_work_free[slot_w]));
    }
}

}  // namespace
}  // namespace gs
