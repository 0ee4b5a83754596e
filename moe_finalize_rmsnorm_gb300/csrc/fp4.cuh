// Device helpers of the 4-bit floating point kernels: E2M1 values (0, 0.5, 1, 1.5, 2, 3,
// 4, 6 and their negatives) and their blocks' scales.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp4.h"

namespace mf {

// Eight values to E2M1, nearest, ties to the even code, beyond 6 to 6; value i in bits
// 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t to_e2m1(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight E2M1 values to pairs of FP16 (exact): value 2 i in the low half of h[i].
__device__ __forceinline__ void from_e2m1(uint32_t q, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
}

// A scale in FP32: E8M0 is an exponent field (0 stands for 2^-127, 255 for NaN), E4M3 is
// read without its sign.
template <int FORMAT>
__device__ __forceinline__ float scale_of(uint32_t byte) {
    if (FORMAT == kMx)
        return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte & 0x7f), __NV_E4M3);
    return __half2float(__half(h));
}

}  // namespace mf
