// Device helpers shared by the expert-layer kernels.
#pragma once

#include "common.cuh"

namespace mf {

// Rows [lo, hi) of expert e.  The offsets are device data that the host cannot
// check, so they are brought into [0, rows] and into order: offsets that do
// not ascend give wrong rows, never an access outside the buffers.
__device__ __forceinline__ void expert_rows(const int32_t *offsets, int e, int rows, int &lo,
                                            int &hi) {
    lo = min(max(__ldg(offsets + e), 0), rows);
    hi = min(max(__ldg(offsets + e + 1), lo), rows);
}

}  // namespace mf
