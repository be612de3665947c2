// gs_attention.cuh -- what the attention kernels share: the bounds of the sequences of a
// ragged batch, the block's tile among them, the mask's row limits, and the tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gs_device.cuh"
#include "gs_tensor.cuh"

namespace gs {

constexpr int kTileRows = 128;                 // rows of every product
constexpr int kBlockCols = 64;                 // values of a 128-byte row in shared memory
constexpr uint32_t kBlockBytes = kTileRows * 128;  // 128 rows x 64 values

struct HeadView {
    __nv_bfloat16* p;
    int64_t ts, hs;
    __device__ __forceinline__ __nv_bfloat16* row(int64_t t, int h) const {
        return p + t * ts + h * hs;
    }
};

// The bounds of a sequence, cut to the arrays.
struct Sequence {
    int64_t q0, k0;
    int n, m;  // queries, keys
};

// how many keys query i of a sequence sees
__device__ __forceinline__ int seen_keys(int i, int n, int m, bool causal) {
    return causal ? min(m, max(0, i + 1 + m - n)) : m;
}

// A block's place: `rows` queries (or keys) of one sequence and a head; and the sequence.
struct Place {
    int b, tile, head;
    Sequence sq;
};

struct Batch {
    const int32_t *cu_q, *cu_k;
    int64_t tq, tk;
    int batch;
    bool causal;
};

// the bounds of sequence b, cut to the arrays: all four offsets are read at once
__device__ __forceinline__ Sequence sequence(const Batch& v, int b) {
    Sequence s{0, 0, (int)v.tq, (int)v.tk};
    if (v.cu_q) {
        const int q0 = __ldg(v.cu_q + b), q1 = __ldg(v.cu_q + b + 1);
        const int k0 = __ldg(v.cu_k + b), k1 = __ldg(v.cu_k + b + 1);
        s.q0 = min(max(q0, 0), (int)v.tq);
        s.n = min(max(q1, (int)s.q0), (int)v.tq) - (int)s.q0;
        s.k0 = min(max(k0, 0), (int)v.tk);
        s.m = min(max(k1, (int)s.k0), (int)v.tk) - (int)s.k0;
    }
    return s;
}

// a lane's sequence to the whole warp
__device__ __forceinline__ Sequence from_lane(const Sequence& s, int lane) {
    const unsigned all = 0xffffffffu;
    return {__shfl_sync(all, (int)s.q0, lane), __shfl_sync(all, (int)s.k0, lane),
            __shfl_sync(all, s.n, lane), __shfl_sync(all, s.m, lane)};
}

// How many of a sequence's tiles cost at least c (c >= 1), cost being the 128-row tiles of
// the other side that a tile meets.  Tiles of queries cost more towards the sequence's end
// under the causal mask, tiles of keys towards its start.  (Tokens are at most 2^30: nothing
// here leaves 32 bits.)
template <bool kKeys>
__device__ __forceinline__ int tiles_from(int n, int m, int rows, bool causal, int c) {
    const int of = kKeys ? m : n, other = kKeys ? n : m;
    const int tiles = (of + rows - 1) / rows;
    const int most = (other + kTileRows - 1) / kTileRows;
    if (c > most) return 0;
    if (!causal) return tiles;
    if (kKeys) {
        // the tile at `key` meets most - max(0, key + n - m) / 128 tiles of queries
        const int y = (most - c + 1) * kTileRows + m - n;
        return y <= 0 ? 0 : min(tiles, (y + rows - 1) / rows);
    }
    // the tile up to query e (exclusive) meets ceil((e + m - n) / 128) tiles of keys
    const int x = (c - 1) * kTileRows + n - m;
    return n <= x ? 0 : tiles - max(0, x) / rows;
}

// By one whole warp: block `id` of the batch's tiles and heads, costliest first where costs
// differ, so that the last blocks to start are short.  False beyond the last one.  Batches
// of more than 32 sequences go sequence by sequence instead, from the last; blocks in between
// may be left without a tile.
template <bool kKeys>
__device__ __forceinline__ bool find_place(const Batch& v, int rows, int heads, int id, Place* at) {
    if (v.batch == 1) {
        const Sequence s = sequence(v, 0);
        const int tiles = ((kKeys ? s.m : s.n) + rows - 1) / rows;
        at->b = 0;
        at->sq = s;
        if (v.causal) {
            const int rank = id / heads;
            at->head = id - rank * heads;
            at->tile = kKeys ? rank : tiles - 1 - rank;
            return rank < tiles;
        }
        // head by head: its keys and values stay in L2 (16,320 tokens x 16 heads x 128 took
        // 8 % longer with the heads in turn)
        at->head = tiles > 0 ? id / tiles : heads;
        at->tile = id - at->head * tiles;
        return at->head < heads;
    }
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    int rank = id / heads;
    at->head = id - rank * heads;
    if (v.batch <= 32) {
        Sequence s{};
        if (lane < v.batch) s = sequence(v, lane);
        const int tiles = ((kKeys ? s.m : s.n) + rows - 1) / rows;
        if (rank >= (int)__reduce_add_sync(all, tiles)) return false;
        // the largest cost that more than `rank` tiles reach (every tile reaches 0)
        int lo = 0;
        int hi = (int)__reduce_max_sync(all, ((kKeys ? s.n : s.m) + kTileRows - 1) / kTileRows);
        while (lo < hi) {
            const int c = (lo + hi + 1) >> 1;
            const int from = tiles_from<kKeys>(s.n, s.m, rows, v.causal, c);
            if ((int)__reduce_add_sync(all, from) > rank)
                lo = c;
            else
                hi = c - 1;
        }
        const int reach = lo == 0 ? tiles : tiles_from<kKeys>(s.n, s.m, rows, v.causal, lo);
        const int above = tiles_from<kKeys>(s.n, s.m, rows, v.causal, lo + 1);
        rank -= (int)__reduce_add_sync(all, above);
        int sum = reach - above;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(all, sum, o);
            if (lane >= o) sum += u;
        }
        const int l = __ffs(__ballot_sync(all, sum > rank)) - 1;
        const int within = rank - (sum - (reach - above));
        const int tile = kKeys ? above + within : tiles - reach + within;
        at->b = l;
        at->tile = __shfl_sync(all, tile, l);
        at->sq = from_lane(s, l);
        return true;
    }
    // A sequence that starts at token t has the slots from t / rows + b on.  They hold its tiles:
    // ceil(n / rows) <= (t + n) / rows + 1 - t / rows.  So a slot's sequence is found without the
    // lengths of those before it, in as many rounds as the batch has powers of 32.
    const int32_t* cu = kKeys ? v.cu_k : v.cu_q;
    const int most = (int)(kKeys ? v.tk : v.tq);
    const auto first_slot = [&](int b) { return min(max(__ldg(cu + b), 0), most) / rows + b; };
    const int slot = most / rows + v.batch - 1 - rank;
    int lo = 0, hi = v.batch;  // the last sequence that starts at the slot or before
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, b = lo + lane * step;
        const unsigned upto = __ballot_sync(all, b < hi && first_slot(b) <= slot);
        if (upto) lo += (31 - __clz(upto)) * step;
        hi = min(hi, lo + step);
    }
    const Sequence s = sequence(v, lo);
    const int tiles = ((kKeys ? s.m : s.n) + rows - 1) / rows, within = slot - first_slot(lo);
    at->b = lo;
    at->tile = kKeys ? tiles - 1 - within : within;
    at->sq = s;
    return within >= 0 && within < tiles;
}

// an upper bound of the tiles of a batch (of several sequences: the slots of find_place)
inline int64_t tiles_at_most(int64_t tokens, int rows, int batch) {
    return batch > 1 ? tokens / rows + batch : (tokens + rows - 1) / rows;
}

// By one whole warp: zeros in rows first..127 of a tile (blocks of 64 columns).
template <int kBlocks>
__device__ __forceinline__ void zero_rows(char* tile, int first) {
    const int lane = threadIdx.x & 31;
    const int words = (kTileRows - first) * 8;
#pragma unroll
    for (int c = 0; c < kBlocks; ++c)
        for (int i = lane; i < words; i += 32)
            *reinterpret_cast<uint4*>(tile + c * kBlockBytes + first * 128 + i * 16) =
                make_uint4(0, 0, 0, 0);
}

// Device address of the count of blocks in which a bounded wait of an attention kernel gave up.
cudaError_t gave_up_word(unsigned int** word);

// Tensor map of a [tokens][heads][dim] array: tiles of 128 tokens of one head, 64 values
// wide under the 128-byte swizzle; zeros beyond the array.  The map's outer dimensions go
// by ascending stride; *swapped says that tokens come before heads.
cudaError_t head_map(CUtensorMap* map, const void* data, int64_t ts, int64_t hs, int64_t tokens,
                     int heads, int dim, bool* swapped);

__device__ __forceinline__ void load_block(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                           int x, int head, int64_t token, bool swapped) {
    if (swapped)
        tma_load(dst, map, bar, x, (int)token, head);
    else
        tma_load(dst, map, bar, x, head, (int)token);
}

// a tile of kBlocks blocks of 64 columns
template <int kBlocks>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                          int head, int64_t token, bool swapped) {
#pragma unroll
    for (int c = 0; c < kBlocks; ++c)
        load_block(dst + c * kBlockBytes, map, bar, c * kBlockCols, head, token, swapped);
}

}  // namespace gs
