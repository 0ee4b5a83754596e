// Rows in chunks of eight values (16 bytes of BF16, 32 of FP32): chunks and their store for
// the permutation's row sum, the store for 4-bit values on their way back; and the load
// that reads or not, and routing weights, for the way into expert order and back, too.
#pragma once

#include "common.cuh"
#include "experts.h"

namespace mf {

// The load of common.cuh's ld_nc_na_16, or zeros (p is not read): no branch between
// the loads of several rows.
__device__ __forceinline__ uint4 ld_nc_na_16_if(const void *p, bool read) {
    uint4 r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
        : "l"(p), "r"(uint32_t{read}));
    return r;
}

template <bool FP32>
struct Chunk8 {
    uint4 v[FP32 ? 2 : 1];
    __device__ void load(const void *rows, int64_t at, bool read) {
        const uint8_t *p = static_cast<const uint8_t *>(rows) + at * (FP32 ? 4 : 2);
        v[0] = ld_nc_na_16_if(p, read);
        if (FP32) v[FP32 ? 1 : 0] = ld_nc_na_16_if(p + 16, read);
    }
    __device__ void get(float (&f)[8]) const {
        if (FP32) {
            const uint4 &a = v[0], &b = v[FP32 ? 1 : 0];
            f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
            f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
            f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
            f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
        } else {
            unpack8(v[0], f);
        }
    }
};

// Eight values to chunk `at` (an element) of BF16 or FP32 rows, rounded once.
template <bool FP32>
__device__ __forceinline__ void store8(void *rows, int64_t at, const float (&f)[8]) {
    if (FP32) {
        float *o = static_cast<float *>(rows) + at;
        st_cs_16(o, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                               __float_as_uint(f[3])));
        st_cs_16(o + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]),
                                   __float_as_uint(f[6]), __float_as_uint(f[7])));
    } else {
        st_cs_16(static_cast<__nv_bfloat16 *>(rows) + at, pack8_rn(f));
    }
}

// Routing weight of a slot.
__device__ __forceinline__ float routing_weight(const void *weights, int kind, int64_t slot) {
    switch (kind) {
        case kRoutingFp32: return __ldg(static_cast<const float *>(weights) + slot);
        case kRoutingBf16:
            return __uint_as_float(
                uint32_t{__ldg(static_cast<const unsigned short *>(weights) + slot)} << 16);
        case kRoutingPacked:
            return bf16_lo(__ldg(static_cast<const uint32_t *>(weights) + slot));
        default: return 1.f;
    }
}

}  // namespace mf
