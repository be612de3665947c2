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

__device__ __forceinline__ void cut(const int32_t* cu, int b, int64_t tokens, int64_t* at, int* n) {
    if (!cu) {
        *at = 0;
        *n = (int)tokens;
        return;
    }
    const int64_t a = min64(max64((int64_t)__ldg(cu + b), 0), tokens);
    const int64_t e = min64(max64((int64_t)__ldg(cu + b + 1), a), tokens);
    *at = a;
    *n = (int)(e - a);
}

// By one whole warp: the sequence and the tile of `rows` rows in it that are number
// `target` of the batch's tiles, counted from the last tile of the last sequence (under
// the causal mask the tiles at a sequence's end have the most work and go first).  False
// beyond the last tile.
__device__ __forceinline__ bool find_tile(const int32_t* cu, int batch, int64_t tokens, int rows,
                                          int target, int* b_out, int* tile_out) {
    if (!cu) {
        const int tiles = (int)((tokens + rows - 1) / rows);
        *b_out = 0;
        *tile_out = tiles - 1 - target;
        return target < tiles;
    }
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int base = 0; base < batch; base += 32) {
        const int b = batch - 1 - base - lane;
        int tiles = 0;
        if (b >= 0) {
            int64_t at;
            int n;
            cut(cu, b, tokens, &at, &n);
            tiles = (n + rows - 1) / rows;
        }
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, before + sum > target);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int upto = __shfl_sync(0xffffffffu, sum, l);
            *b_out = batch - 1 - base - l;
            *tile_out = before + upto - 1 - target;
            return true;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}

// how many keys query i of a sequence sees
__device__ __forceinline__ int seen_keys(int i, int n, int m, bool causal) {
    return causal ? min(m, max(0, i + 1 + m - n)) : m;
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

// Device address of the word that is set when a bounded wait of an attention kernel gave up.
cudaError_t gave_up_word(unsigned int** word);

// Tensor map of a [tokens][heads][dim] array: tiles of 128 tokens of one head, 64 values
// wide under the 128-byte swizzle; zeros beyond the array.  The map's outer dimensions go
// by ascending stride; *swapped says that tokens come before heads.
cudaError_t head_map(CUtensorMap* map, const void* data, int64_t ts, int64_t hs, int64_t tokens,
                     int heads, int dim, bool* swapped);

struct MapSwaps {
    bool q, k, v, o;
};

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
