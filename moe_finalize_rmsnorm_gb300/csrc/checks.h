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

// Rows of `width` bytes, `stride` bytes apart.
struct ByteRows {
    const void *p;
    int64_t rows, stride, width;
    int64_t extent() const {  // (2^31 rows may lie 2^36 bytes apart)
        if (rows <= 0) return 0;
        const __int128 e = static_cast<__int128>(rows - 1) * stride + width;
        return e < INT64_MAX ? static_cast<int64_t>(e) : INT64_MAX;
    }
};

// Whether two sets of rows share a byte.  Columns side by side in rows of one stride do not;
// rows of different strides count as sharing what lies between their ends.
inline bool overlap(const ByteRows &a, const ByteRows &b) {
    if (!overlap(a.p, a.extent(), b.p, b.extent())) return false;
    if (a.rows == 1 && b.rows == 1) return true;
    const int64_t stride = a.rows > 1 ? a.stride : b.stride;
    if (b.rows > 1 && b.stride != stride) return true;
    const int64_t from = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) -
                                              reinterpret_cast<uintptr_t>(a.p));
    const int64_t at = (from % stride + stride) % stride;  // b's columns, in a's rows
    return at < a.width || at + b.width > stride;
}

}  // namespace mf
