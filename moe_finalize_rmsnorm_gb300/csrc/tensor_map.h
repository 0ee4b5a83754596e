// Host: tensor maps for the copies of tiles (TMA).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mf {

// Find the driver's encoder (once, before the first map; not thread-safe by itself).
cudaError_t find_encoder();

// Map of a row-major tensor of `rank` 2 or 3: sizes fastest first, byte strides of
// the slower dimensions, boxes of `columns` (128 bytes, stored with the 128-byte
// swizzle) by `rows`; what lies outside the tensor arrives as zeros.  False if the
// driver refuses it.
bool encode_map(CUtensorMap *m, CUtensorMapDataType type, const void *p, int rank,
                const cuuint64_t (&sizes)[3], const cuuint64_t (&strides)[2], int columns, int rows);

}  // namespace mf
