// gs_attention_fwd.cuh -- what the attention forward's kernels share: the shapes in shared and
// tensor memory, the cutting of blocks' keys into pieces and the joining of the pieces.
#pragma once

#include "gs_attention.cuh"

namespace gs {
namespace {

constexpr int kSoftmaxWarps = 8;
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
    int most_keys;  // key tiles that a block may walk
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
    Window window;  // batch.causal is not set with one: its blocks cost about the same
    float *part_o, *part_lse;  // [pieces][rest][slot_rows][DP], [pieces][rest][slot_rows]
};

// key tiles that query tile t (128 rows) of the block at row0 walks
__device__ __forceinline__ int walked(const Sequence& sq, int row0, int t, bool causal) {
    const int last = min(sq.n, row0 + (t + 1) * kTileRows) - 1;
    return last >= row0 + t * kTileRows
               ? (seen_keys(last, sq.n, sq.m, causal) + kTileRows - 1) / kTileRows
               : 0;
}

// With a window: the walk of both query tiles, each tile's end in it, and the step that the
// second leaves out (-1: none), since it sees no key of the first's first tile.
struct FwdWalk {
    Walk walk;
    int end[2], skip;
};

__device__ __forceinline__ FwdWalk walk_of_block(const Window& w, const Sequence& sq, int row0) {
    FwdWalk f;
    const int last = min(sq.n, row0 + 2 * kTileRows) - 1;
    f.walk = walk_of(w, sq, row0, last);
    const Seen s = seen_by(w, min(last, row0 + kTileRows - 1), sq.n, sq.m);
    f.end[0] = max(0, walk_end(s) - f.walk.first) + f.walk.extra;
    f.end[1] = row0 + kTileRows < sq.n ? f.walk.tiles : 0;
    f.skip = -1;
    if (f.end[1] > 0 && (f.walk.first > 0 || w.sinks == 0) &&  // the sinks lie in tile 0
        seen_by(w, row0 + kTileRows, sq.n, sq.m).lo / kTileRows > f.walk.first)
        f.skip = f.walk.extra;
    return f;
}

// Spread blocks (by one whole warp; lane = sequence): the smallest chunk with which kSms
// blocks suffice, and the place of block or piece `id`.  Pieces of a block are neighbours.
struct Spread {
    int chunk, pieces;  // of the place's sequence
    int piece;          // with `cut`: which one
    int first;          // number of the block's first piece
};

__device__ __forceinline__ bool find_spread(const Batch& v, int heads, int id, bool by_piece,
                                            int most_keys, Place* at, Spread* sp) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    Sequence s{};
    if (lane < v.batch) s = sequence(v, lane);
    const int n = s.n, m = s.m;
    const int blocks = (n + 2 * kTileRows - 1) / (2 * kTileRows) * heads;
    const int keys = min((m + kTileRows - 1) / kTileRows, most_keys);
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

// A split block's rows from its pieces, in the order of the pieces.  DP / 4 lanes a row.
constexpr int kJoinThreads = 256;

template <int DP, bool kWindow>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const FwdParams p) {
    __shared__ Place place;
    __shared__ Spread spread;
    __shared__ int found;
    grid_dep_sync();
    if (threadIdx.x < 32) {
        Place at{};
        Spread sp{p.plan.chunk, p.plan.pieces, 0, (int)blockIdx.x};
        const bool ok = p.plan.spread
                            ? find_spread(p.batch, p.heads, blockIdx.x, false, p.plan.most_keys, &at,
                                          &sp)
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
        const int walks = kWindow ? walk_of_block(p.window, sq, row0).end[r / kTileRows]
                                  : walked(sq, row0, r / kTileRows, p.batch.causal);
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

}  // namespace
}  // namespace gs
