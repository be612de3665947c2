// gs_attention_fwd.cu -- softmax attention, forward, on the tensor cores.
//
//   S = scale Q K^T,  P = exp(S - row maximum),  O = P V / row sum
//
// in one pass over the keys with a running maximum and sum.  A block takes 256 queries of
// one head as two tiles of 128 rows, with the key and value tiles (128 rows) shared by
// both.  A producer warp brings tiles by TMA into a ring, one thread issues the products,
// and four warps per query tile do its softmax, one row a thread: S comes from tensor
// memory, P goes back over it in bfloat16 as the second product's first operand, O stays
// in tensor memory.  While one tile's softmax runs, the tensor cores work on the other's
// products.
//
// The running maximum is stale on purpose: a row's O and sum are rescaled only once its
// maximum has risen by more than 8 (in powers of two), so P stays below 2^8 and the
// rescaling, which has to wait for the last product, is rare.  P is rounded to bfloat16
// for the product; the sum takes the unrounded values in fp32.
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

struct FwdParams {
    int64_t tq, tk;
    int batch, group, dim;
    bool causal, negative, swap_q, swap_k, swap_v;
    float scale, log2_scale;  // |scale|, and with log2(e)
    HeadView o;
    float* lse;
    unsigned int* gave_up;
    const int32_t *cu_q, *cu_k;
};

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attention_fwd_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const FwdParams p) {
    using Sh = FwdShape<DP>;
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bar_q[2], bar_s[2 * Sh::kScores], bar_p[2 * Sh::kScores], bar_o[2], bar_full[Sh::kSlots],
        bar_empty[Sh::kSlots], bar_raw, bar_drain;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    __shared__ int sh_b, sh_tile, sh_found;

    grid_dep_sync();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        int b = 0, tile = 0;
        const bool found =
            find_tile(p.cu_q, p.batch, p.tq, 2 * kTileRows, blockIdx.x, &b, &tile);
        if (lane == 0) sh_b = b, sh_tile = tile, sh_found = found, dead = 0;
    }
    __syncthreads();
    if (!sh_found) return;
    Sequence sq;
    cut(p.cu_q, sh_b, p.tq, &sq.q0, &sq.n);
    cut(p.cu_k, sh_b, p.tk, &sq.k0, &sq.m);
    const int row0 = sh_tile * 2 * kTileRows;  // first query of the block in its sequence
    const int head = blockIdx.y, khead = head / p.group;
    // key tiles that each of the two query tiles walks
    int tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int last = min(sq.n, row0 + (t + 1) * kTileRows) - 1;
        tiles[t] = last >= row0 + t * kTileRows
                       ? (seen_keys(last, sq.n, sq.m, p.causal) + kTileRows - 1) / kTileRows
                       : 0;
    }
    const int most = max(tiles[0], tiles[1]);

    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t smem_kv = smem + 2 * Sh::kTileBytes;
    if (warp == kSoftmaxWarps) {
        tmem_alloc(smem_u32(&tmem_at), 512);
    } else if (threadIdx.x == 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bar_q[t]), 1);
            mbar_init(smem_u32(&bar_o[t]), 1);
        }
        for (int i = 0; i < 2 * Sh::kScores; ++i) {
            mbar_init(smem_u32(&bar_s[i]), 1);
            mbar_init(smem_u32(&bar_p[i]), 4);
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
    const auto order = [&](int j, int t) { return min(j + t, tiles[0]) + min(j, tiles[1]); };
    const auto tmem_s = [&](int x) { return tmem + (x % Sh::kScores) * 128; };
    const auto tmem_o = [&](int t) { return tmem + Sh::kScores * 128 + t * DP; };

    if (warp == kSoftmaxWarps + 1) {
        // ---- the producer: Q, then K and V tiles in turn ----
        if (most > 0) {
            if (elect_one()) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (tiles[t] > 0) {
                        mbar_expect(smem_u32(&bar_q[t]), Sh::kTileBytes);
                        load_tile<Sh::kBlocks>(smem + t * Sh::kTileBytes, &map_q,
                                               smem_u32(&bar_q[t]), head,
                                               sq.q0 + row0 + t * kTileRows, p.swap_q);
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
                const int valid = sq.m - j * kTileRows;
                // values of another sequence behind this one's end: zeros in their place
                const bool mend = is_v && valid < kTileRows && sq.k0 + sq.m < p.tk;
                const uint32_t bar = mend ? smem_u32(&bar_raw) : full;
                if (elect_one()) {
                    mbar_expect(bar, Sh::kTileBytes);
                    load_tile<Sh::kBlocks>(dst, is_v ? &map_v : &map_k, bar, khead,
                                           sq.k0 + (int64_t)j * kTileRows,
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
            if (i < 2 * most) {  // gave up: no copy outlives the block
                for (int t = 0; t < 2; ++t)
                    if (tiles[t] > 0) mbar_drain(smem_u32(&bar_q[t]), 0);
                for (int u = max(0, i - Sh::kSlots); u < i; ++u)
                    mbar_drain(smem_u32(&bar_full[u % Sh::kSlots]), (u / Sh::kSlots) & 1);
            }
        }
    } else if (warp == kSoftmaxWarps) {
        // ---- the products ----
        // By one thread (a whole warp that walks the steps with one thread issuing took 1,414
        // us instead of 1,283 on 16,320 tokens x 16 heads x 128).  A step is a key tile and a
        // query tile; scores run kScores steps ahead of the outputs, so that a query tile's
        // softmax finds its next scores ready.
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
                ok = ok && mbar_wait(smem_u32(&bar_full[ahead.slot]), ahead.phase, &dead);
                if (ahead.j == 0) ok = ok && mbar_wait(smem_u32(&bar_q[ahead.t]), 0, &dead);
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
                ok = mbar_wait(smem_u32(&bar_full[at.slot + 1]), at.phase, &dead) &&
                     mbar_wait(smem_u32(&bar_p[at.t * Sh::kScores + at.bar]), at.turn, &dead);
                if (!ok) break;
                tmem_fence_after();
                const Step s = at;
                product_rows(tmem_o(s.t), tmem_s(s.score), 32, op_v + s.slot * kTileStep, word_o,
                             s.j > 0);
                mma_commit(smem_u32(&bar_o[s.t]));
                if (ahead.j < most) scores();
                if (advance(at)) mma_commit(smem_u32(&bar_empty[s.slot + 1]));
            }
            if (!ok) {  // leave no product in flight
                mma_commit(smem_u32(&bar_drain));
                mbar_drain(smem_u32(&bar_drain), 0);
            }
        }
    } else {
        // ---- softmax: one row a thread ----
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's lanes of tensor memory
        const int i = row0 + t * kTileRows + r;
        const int limit = seen_keys(i, sq.n, sq.m, p.causal);
        const int first_limit =
            seen_keys(row0 + t * kTileRows + (warp & 3) * 32, sq.n, sq.m, p.causal);
        const float sl = p.log2_scale, tau = kStale / sl;
        const uint32_t o_at = tmem_o(t) + lanes;
        float top = -INFINITY;
        float2 sum = make_float2(0.f, 0.f);
        bool ok = true;
        for (int j = 0; j < tiles[t]; ++j) {
            const uint32_t s_at = tmem_s(order(j, t)) + lanes;
            // kScores barriers a query tile: the one of j is used again after P(j) is taken
            ok = mbar_wait(smem_u32(&bar_s[t * Sh::kScores + j % Sh::kScores]),
                           (j / Sh::kScores) & 1, &dead);
            if (!ok) break;
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
            const bool risen = high > top + tau;
            if (__any_sync(0xffffffffu, risen)) {
                const float f = risen ? ex2_approx((top - high) * sl) : 1.f;
                if (risen) top = high;
                sum.x *= f;
                sum.y *= f;
                if (j > 0) {
                    ok = mbar_wait(smem_u32(&bar_o[t]), (j - 1) & 1, &dead);
                    if (!ok) break;
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
        if (ok && tiles[t] > 0) ok = mbar_wait(smem_u32(&bar_o[t]), (tiles[t] - 1) & 1, &dead);
        if (ok) {
            tmem_fence_after();
            const float l = sum.x + sum.y;
            const bool valid = i < sq.n;
            // a row that sees no key: zeros
            const float f = limit > 0 ? 1.f / l : 0.f;
            __nv_bfloat16* out = valid ? p.o.row(sq.q0 + i, head) : nullptr;
#pragma unroll
            for (int c = 0; c < DP; c += 32) {
                uint32_t o[32];
                if (tiles[t] > 0) {
                    tmem_ld32(o, o_at + c);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
                if (!valid) continue;
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    if (c + k >= p.dim) break;
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = __uint_as_float(o[k + 2 * e]) * f;
                        const float b = __uint_as_float(o[k + 2 * e + 1]) * f;
                        w[e] = limit > 0 ? pack_bf16(a, b) : 0u;
                    }
                    *reinterpret_cast<uint4*>(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (valid)
                p.lse[(int64_t)head * p.tq + sq.q0 + i] =
                    limit > 0 ? (fmaf(top, sl, log2f(l))) * 0.69314718055994530942f : -INFINITY;
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (dead && threadIdx.x == 0) *p.gave_up = 1;
    if (warp == kSoftmaxWarps) {
        __syncwarp();
        tmem_fence_after();
        tmem_free(tmem_at, 512);
    }
}

template <int DP>
cudaError_t launch_dim(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       const FwdParams& p, int heads, cudaStream_t st) {
    const cudaError_t e =
        cudaFuncSetAttribute(attention_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)FwdShape<DP>::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t rows = 2 * kTileRows;
    const int64_t tiles = p.cu_q ? p.tq / rows + p.batch : (p.tq + rows - 1) / rows;
    return launch(attention_fwd_kernel<DP>, dim3((unsigned)tiles, (unsigned)heads),
                  dim3(kFwdThreads), FwdShape<DP>::kSmem, st, mq, mk, mv, p);
}

}  // namespace

cudaError_t launch_attention_fwd(const gs_attention_shape& s, const gs_heads& q, const gs_heads& k,
                                 const gs_heads& v, const gs_heads& out, float* lse,
                                 const int32_t* cu_q, const int32_t* cu_k, void* ws,
                                 cudaStream_t st) {
    (void)ws;
    FwdParams p{};
    p.tq = s.tokens_q;
    p.tk = s.tokens_k;
    p.batch = s.batch;
    p.group = s.heads_q / s.heads_k;
    p.dim = s.head_dim;
    p.causal = s.causal != 0;
    p.negative = s.scale < 0.f;
    p.scale = fabsf(s.scale);
    // a zero scale as one too small to matter: masked scores of -infinity stay defined
    p.log2_scale = fmaxf(p.scale * 1.4426950408889634f, 1e-30f);
    p.o = {static_cast<__nv_bfloat16*>(out.data), out.token_stride, out.head_stride};
    p.lse = lse;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
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
    return s.head_dim <= 64 ? launch_dim<64>(mq, mk, mv, p, s.heads_q, st)
                            : launch_dim<128>(mq, mk, mv, p, s.heads_q, st);
}

}  // namespace gs
