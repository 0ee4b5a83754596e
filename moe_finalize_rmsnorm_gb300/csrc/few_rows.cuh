// What the products of few rows per expert share: a warp takes 32 output columns of
// an expert and streams their weights past the rows.
#pragma once

#include "experts.cuh"

namespace mf {

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <typename T>
__device__ __forceinline__ T lds(uint32_t addr) {
    return *reinterpret_cast<const T *>(__cvta_shared_to_generic(addr));
}

// Where a warp is in its sequence of (column block, stage) pairs.
struct Cursor {
    int item;
    int stage;  // of the item's spans
    int expert, n0, row0, rows;
};

// Host: warps to a column block, as many as make the longest warp's work shortest,
// counted in stages, a block's beginning and end as two.  `blocks`: column blocks at most
// (the experts' sizes are known on the device only), `spans`: stages of one.  Of 1, 2, 3, 4,
// 5 and 8 warps forced it took the fastest in eight of eight shapes (4-bit, 8 x 4096 x 4096:
// 21.9, 18.3, 21.3, 18.7, 22.6 and 21.1 us; 20003 x 7168: 37, 23.5, 20.9, 24.9, 23.2, 24.3).
inline int warps_of_block(int64_t blocks, int spans, int warps, int num_sms) {
    int share = 1;
    int64_t best = INT64_MAX;
    for (int w : {1, 2, 3, 4, 5, 6, 8, 12, 16}) {
        if (w > spans || w > warps) break;
        const int64_t at_once = int64_t{num_sms} * (warps / w);
        const int64_t cost = (blocks + at_once - 1) / at_once * ((spans + w - 1) / w + 2);
        if (cost < best) {
            best = cost;
            share = w;
        }
    }
    return share;
}

// The first column block of a warp, with `at_once` blocks to a CTA: blocks that lie
// together to one CTA's warps (they read the same rows of x), unless there are so few
// that this would leave CTAs without.  A warp that is left over gets none (`items`).
__device__ __forceinline__ int first_item(int block, int at_once, int items) {
    if (block >= at_once) return items;
    return items >= 4 * static_cast<int>(gridDim.x) * at_once ? blockIdx.x * at_once + block
                                                              : blockIdx.x + gridDim.x * block;
}

}  // namespace mf
