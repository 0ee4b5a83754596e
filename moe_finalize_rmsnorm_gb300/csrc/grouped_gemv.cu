// Products of few rows per expert with 4-bit weights and group scales.
#include "experts.cuh"
#include "experts.h"

namespace mf {
namespace {

// One warp per output column n of an expert, one row after the other.  Each
// group's sum of (q - z) x is scaled once, in FP32.
__global__ void __launch_bounds__(256) gemv_int4_simple_kernel(GemvArgs a) {
    pdl_wait();
    const int lane = threadIdx.x % 32;
    const int n = blockIdx.x * 8 + threadIdx.x / 32;
    const int e = blockIdx.y;
    int lo = 0, hi = static_cast<int>(a.rows);
    if (a.offsets) expert_rows(a.offsets, e, static_cast<int>(a.rows), lo, hi);
    if (n >= a.n) return;
    const int64_t line = int64_t{e} * a.n + n;
    const int groups = a.k / a.group;
    const uint8_t *w = a.w + line * (a.k / 2);
    for (int r = lo; r < hi; ++r) {
        const int64_t row = a.row_index ? a.row_index[r] : r;
        float acc = 0.f;
        if (row >= 0 && row < a.x_rows) {
            const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x) + row * a.x_ld;
            for (int g = lane; g < groups; g += 32) {
                const float z = a.zeros ? float(a.zeros[line * groups + g] & 15) : 8.f;
                const float sc =
                    a.scale_fp32
                        ? static_cast<const float *>(a.scales)[line * groups + g]
                        : __bfloat162float(
                              static_cast<const __nv_bfloat16 *>(a.scales)[line * groups + g]);
                float part = 0.f;
                for (int c = g * a.group; c < (g + 1) * a.group; c += 2) {
                    const int b = w[c / 2];
                    part = fmaf((b & 15) - z, __bfloat162float(x[c]), part);
                    part = fmaf((b >> 4) - z, __bfloat162float(x[c + 1]), part);
                }
                acc = fmaf(sc, part, acc);
            }
        }
        acc = warp_sum(acc);
        if (lane == 0) {
            if (a.out_fp32)
                static_cast<float *>(a.out)[r * a.out_ld + n] = acc;
            else
                static_cast<__nv_bfloat16 *>(a.out)[r * a.out_ld + n] = __float2bfloat16_rn(acc);
        }
    }
}

}  // namespace

cudaError_t launch_grouped_gemv_int4(const GemvArgs &a, cudaStream_t s) {
    return launch_ex(gemv_int4_simple_kernel, dim3((a.n + 7) / 8, a.num_experts), dim3(256), 0, s,
                     1, a.programmatic, a);
}

}  // namespace mf
