// gs_attention.cu -- host parts that the attention kernels share: tensor maps, the size of
// the workspace, and the count of blocks in which a wait gave up.
#include <cuda_runtime.h>

#include <cstdint>

#include "gs_attention.cuh"
#include "gs_internal.h"
#include "gs_tokens.h"

namespace gs {
namespace {

__device__ unsigned int g_gave_up;  // only ever counted up: every thread of the host compares

// test only: a warp's bounded wait in which the last lane alone waits for a phase that does not
// come, the others for the one before it, which is done; reported if the warp gave up as one
__global__ void waiting_kernel(unsigned int* gave_up) {
    grid_dep_sync();
    __shared__ uint64_t bar;
    __shared__ volatile int dead;
    if (threadIdx.x == 0) {
        dead = 0;
        mbar_init(smem_u32(&bar), 1);
        fence_barrier_init();
    }
    __syncthreads();
    const bool ok = mbar_wait(smem_u32(&bar), threadIdx.x == 31 ? 0 : 1, &dead);
    if (!ok && threadIdx.x == 0) atomicAdd(gave_up, 1u);
}

}  // namespace

cudaError_t gave_up_word(unsigned int** word) {
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_gave_up);
    *word = static_cast<unsigned int*>(p);
    return e;
}

cudaError_t attention_gave_up(cudaStream_t st, bool* gave_up) {
    // what this thread has been told of: a report to one thread takes it from no other
    constexpr int kDevices = 64;
    static thread_local unsigned int told[kDevices];
    unsigned int *word = nullptr, count = 0;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess && device >= kDevices) e = cudaErrorInvalidDevice;
    if (e == cudaSuccess) e = gave_up_word(&word);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(&count, word, sizeof(count), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return e;
    *gave_up = count != told[device];
    told[device] = count;
    return cudaSuccess;
}

cudaError_t head_map(CUtensorMap* map, const void* data, int64_t ts, int64_t hs, int64_t tokens,
                     int heads, int dim, bool* swapped) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    // the driver's function, looked up once (a function's address does not change)
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return cudaErrorNotSupported;
    *swapped = ts < hs;
    const cuuint64_t size[3] = {(cuuint64_t)dim, (cuuint64_t)(*swapped ? tokens : heads),
                                (cuuint64_t)(*swapped ? heads : tokens)};
    const cuuint64_t stride[2] = {(cuuint64_t)(*swapped ? ts : hs) * 2,
                                  (cuuint64_t)(*swapped ? hs : ts) * 2};
    const cuuint32_t box[3] = {kBlockCols, *swapped ? kTileRows : 1u, *swapped ? 1u : kTileRows};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(data),
                              size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

size_t attention_workspace_bytes(int64_t tokens_q, int64_t tokens_k, int batch, int heads_q,
                                 int heads_k, int head_dim) {
    const size_t fwd = attention_fwd_workspace_bytes(tokens_q, tokens_k, batch, heads_q, head_dim);
    const size_t bwd =
        attention_bwd_workspace_bytes(tokens_q, tokens_k, batch, heads_q, heads_k, head_dim);
    return (fwd > bwd ? fwd : bwd) / 256 * 256 + 512;
}

}  // namespace gs

// Not part of the C ABI (tests): runs the attention kernels' bounded wait out on the product's
// own wait, so that gs_attention_status has something to report.
extern "C" gs_status gs_test_attention_wait(void* stream) {
    unsigned int* word = nullptr;
    cudaError_t e = gs::gave_up_word(&word);
    if (e == cudaSuccess)
        e = gs::launch(gs::waiting_kernel, dim3(1), dim3(32), 0, (cudaStream_t)stream, word);
    return e == cudaSuccess ? GS_OK : GS_ERR_CUDA;
}
