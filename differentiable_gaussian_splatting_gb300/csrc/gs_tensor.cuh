// gs_tensor.cuh -- the tensor-core vocabulary of the attention kernels (sm_103a):
// mbarriers with bounded waits, TMA tile loads, tensor memory, and the 128-row
// tcgen05 products of bfloat16 tiles.
//
// Tiles lie in shared memory as TMA writes them under the 128-byte swizzle: rows of
// 64 bfloat16 (128 bytes), eight rows to a 1,024-byte atom, a tile of 128 values a
// row as two such blocks of columns one after the other.  The same bytes serve as an
// operand whose rows run along the product's outer dimension (contracted along the
// columns) and as one contracted along the rows; only the descriptor differs.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace gs {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

// ---------------------------------------------------------------------------
// mbarriers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// A wait gives up after this many clocks (over a second), tells the block through
// `dead` and returns false; the block then drains its copies and products and ends.
constexpr long long kWaitClocks = 4000000000ll;

__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* dead) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (*dead) return false;
        if (clock64() - t0 > kWaitClocks) {
            *dead = 1;
            return false;
        }
    }
    return true;
}
// by one thread
__device__ __forceinline__ bool mbar_wait_one(uint32_t bar, uint32_t parity, volatile int* dead) {
    return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, dead);
}
// By a whole warp, whose lanes go on or give up together: a lane may find the phase done just as
// another's limit runs out, and what follows is in step.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    return __all_sync(0xffffffffu, mbar_wait_one(bar, parity, dead));
}
// By a whole warp that goes on all the same where the wait has given up, with whatever it finds:
// its lanes stay together without a vote's answer to branch on (8,160 tokens x 16 heads on 4 x
// 64: forward 265 instead of 272 us, gradient 846 instead of 863).  What follows may only compute
// and arrive; copies and products are issued, and results written, behind the waits above or a
// look at `dead`.
__device__ __forceinline__ void mbar_pass(uint32_t bar, uint32_t parity, volatile int* dead) {
    mbar_wait_one(bar, parity, dead);
    __syncwarp();
}
// by a whole warp, all of whose lanes get the same answer
__device__ __forceinline__ bool any_dead(volatile int* dead) {
    return __any_sync(0xffffffffu, *dead != 0);
}

// A block ends when its own copies and products have: whoever issued them waits for them last
// of all, with the same limit, whether or not a wait of the block has given up.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity) && clock64() - t0 < kWaitClocks) {
    }
}
// the last of `items` copies that went round a ring of kSlots barriers
template <int kSlots>
__device__ __forceinline__ void drain_ring(const uint64_t* full, int items) {
    for (int u = max(0, items - kSlots); u < items; ++u)
        mbar_drain(smem_u32(&full[u % kSlots]), (u / kSlots) & 1);
}

// writes of ordinary stores become visible to TMA and the tensor cores
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// ---------------------------------------------------------------------------
// TMA
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                         int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------------------
// tensor memory
// ---------------------------------------------------------------------------
// by one whole warp; the address goes to shared memory
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define GS_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                    "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define GS_V8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                    "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of the warp's 32 lanes: thread = lane, register = column
__device__ __forceinline__ void tmem_ld32(uint32_t* r, uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : GS_R8(r, 0), GS_R8(r, 8), GS_R8(r, 16), GS_R8(r, 24)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31};" ::GS_V8(r, 0),
        GS_V8(r, 8), GS_V8(r, 16), GS_V8(r, 24), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t* r, uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : GS_R8(r, 0), GS_R8(r, 8)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15};" ::GS_V8(r, 0),
        GS_V8(r, 8), "r"(addr)
        : "memory");
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// Instruction word of a bfloat16 product with fp32 results: M x N, the second operand
// contracted along its rows (kRowsB) or its columns, the first negated or not.
__host__ __device__ constexpr uint32_t mma_word(int M, int N, bool rows_a, bool rows_b) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)rows_a << 15) |
           ((uint32_t)rows_b << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kNegateA = 1u << 13;

// Descriptors of swizzled operands: their low words, address and the distance of their
// blocks of 64 columns (128 rows each; not read where the product is contracted along the
// columns).  The high word is the same for all: atoms of eight rows follow each other
// (1,024 bytes), 128-byte swizzle.  In 32 bits the address steps are single additions; with
// 64-bit descriptors the issuing thread held up the forward by 2 %.
constexpr uint32_t kOperandHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t operand_columns(uint32_t addr) {
    return ((addr & 0x3ffff) >> 4) | (1u << 16);
}
__device__ __forceinline__ uint32_t operand_rows(uint32_t addr) {
    return ((addr & 0x3ffff) >> 4) | ((128u * 128u >> 4) << 16);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t word,
                                       bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(word), "r"((uint32_t)add), "r"(kOperandHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t word,
                                       bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(word), "r"((uint32_t)add), "r"(kOperandHigh)
        : "memory");
}
// the barrier gets one arrival when all products issued so far by this thread are done
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// D[128 x N] (+)= A B^T over kDim columns, both operands contracted along their columns:
// A 128 rows, B N rows, blocks of 64 columns of 128 rows each.  The steps along the columns
// add to the descriptors' address.
template <int kDim>
__device__ __forceinline__ void product_columns(uint32_t d, uint32_t a, uint32_t b, uint32_t word,
                                                bool add) {
#pragma unroll
    for (int k = 0; k < kDim / 16; ++k) {
        const uint32_t in = (k >> 2) * (128 * 128 / 16) + (k & 3) * 2;
        mma_ss(d, a + in, b + in, word, add || k > 0);
    }
}

// D[128 x N] (+)= A B with A [128 x 128] in tensor memory (two bfloat16 a column) and B
// contracted along its 128 rows.  A's halves of 64 contracted rows lie `half` columns apart.
__device__ __forceinline__ void product_rows(uint32_t d, uint32_t a, uint32_t half, uint32_t b,
                                             uint32_t word, bool add) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
        mma_ts(d, a + (k >> 2) * half + (k & 3) * 8, b + k * 128, word, add || k > 0);
}

// ---------------------------------------------------------------------------
// arithmetic
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace gs
