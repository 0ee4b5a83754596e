// Argument checks that the C entry points of the expert layer share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_finalize.h"

namespace mf {

constexpr int64_t kMaxRows = 0x7fffffffLL - 1024;  // row numbers and tile ends stay in int32
constexpr int32_t kMaxWidth = 1 << 20;             // columns of a matrix

inline mf_status from_launch(cudaError_t e) { return e == cudaSuccess ? MF_OK : MF_ERR_CUDA; }

inline bool value_dtype(mf_dtype d) { return d == MF_DTYPE_BF16 || d == MF_DTYPE_FP32; }

// Row strides of the 16-byte kernels: at least the row, a multiple of 8 elements.
inline bool row_stride_ok(int64_t stride, int64_t width) {
    return stride >= width && stride % 8 == 0 && stride < (int64_t{1} << 36);
}

// Whether two buffers share a byte (an empty one shares none).
inline bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    if (a_bytes <= 0 || b_bytes <= 0) return false;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + static_cast<uintptr_t>(b_bytes) && q < p + static_cast<uintptr_t>(a_bytes);
}

}  // namespace mf
