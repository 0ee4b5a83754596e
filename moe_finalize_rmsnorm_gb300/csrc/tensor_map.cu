// Tensor maps, by the driver's encoder (host code only).
#include "tensor_map.h"

#include <atomic>

namespace mf {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Two threads may look it up at once, each under another family's lock: both store the same.
std::atomic<EncodeFn> g_encode{nullptr};

}  // namespace

bool encode_map(CUtensorMap *m, CUtensorMapDataType type, const void *p, int rank,
                const cuuint64_t (&sizes)[3], const cuuint64_t (&strides)[2], int columns,
                int rows) {
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(columns), static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    const EncodeFn encode = g_encode.load(std::memory_order_acquire);
    const auto encoded = [&] {
        return encode(m, type, rank, const_cast<void *>(p), sizes, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = encoded();
    // The driver wants a context, which a thread has only after some call of the runtime's:
    // setting the device, the same one, is such a call.
    int dev = 0;
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess &&
        cudaSetDevice(dev) == cudaSuccess)
        r = encoded();
    return r == CUDA_SUCCESS;
}

cudaError_t find_encoder() {
    if (g_encode.load(std::memory_order_acquire)) return cudaSuccess;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    g_encode.store(reinterpret_cast<EncodeFn>(fn), std::memory_order_release);
    return cudaSuccess;
}

}  // namespace mf
