// Matrix products grouped by expert: forward, and the gradients of the rows
// and of the weights.
#include "experts.cuh"
#include "experts.h"

namespace mf {
namespace {

constexpr int kTile = 64, kStep = 16;

// One 64 x 64 tile of an expert's product per CTA, FP32 multiply-adds, 4 x 4
// results per thread.  Result (i, j) = sum_c A(i, c) B(j, c):
//   forward  i = row r, j = n, c = k:  A = x,    B = W[e]
//   dgrad    i = row r, j = k, c = n:  A = dy,   B = W[e] transposed
//   wgrad    i = n,     j = k, c = r:  A = dy^T, B = x^T
template <int KIND>
__global__ void __launch_bounds__(256) grouped_gemm_simple_kernel(GroupedArgs a) {
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    pdl_wait();
    const int e = blockIdx.z;
    int lo, hi;
    expert_rows(a.offsets, e, static_cast<int>(a.rows), lo, hi);
    const int m = hi - lo;
    const int I = KIND == kWgrad ? a.n : m;
    const int J = KIND == kForward ? a.n : a.k;
    const int C = KIND == kForward ? a.k : KIND == kDgrad ? a.n : m;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x);
    const __nv_bfloat16 *dy = static_cast<const __nv_bfloat16 *>(a.dy);
    const __nv_bfloat16 *w =
        KIND == kWgrad ? nullptr : static_cast<const __nv_bfloat16 *>(a.w) + e * a.w_expert;
    auto x_at = [&](int r, int c) -> float {
        const int64_t row = a.row_index ? a.row_index[lo + r] : lo + r;
        if (row < 0 || row >= a.x_rows) return 0.f;
        return __bfloat162float(x[row * a.x_ld + c]);
    };
    auto dy_at = [&](int r, int c) { return __bfloat162float(dy[(lo + r) * a.dy_ld + c]); };
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int j0 = blockIdx.x * kTile;
    for (int i0 = blockIdx.y * kTile; i0 < I; i0 += gridDim.y * kTile) {
        float acc[4][4] = {};
        for (int c0 = 0; c0 < C; c0 += kStep) {
            for (int t = threadIdx.x; t < kTile * kStep; t += 256) {
                const int c = KIND == kWgrad ? t / kTile : t % kStep;
                const int i = KIND == kWgrad ? t % kTile : t / kStep;
                const bool in_c = c0 + c < C;
                float v = 0.f, u = 0.f;
                if (in_c && i0 + i < I)
                    v = KIND == kForward ? x_at(i0 + i, c0 + c)
                        : KIND == kDgrad ? dy_at(i0 + i, c0 + c)
                                         : dy_at(c0 + c, i0 + i);
                if (in_c && j0 + i < J)
                    u = KIND == kForward ? __bfloat162float(w[(j0 + i) * a.w_ld + c0 + c])
                        : KIND == kDgrad ? __bfloat162float(w[(c0 + c) * a.w_ld + j0 + i])
                                         : x_at(c0 + c, j0 + i);
                as[c][i] = v;
                bs[c][i] = u;
            }
            __syncthreads();
            for (int c = 0; c < kStep; ++c)
                for (int p = 0; p < 4; ++p)
                    for (int q = 0; q < 4; ++q)
                        acc[p][q] = fmaf(as[c][ty + 16 * p], bs[c][tx + 16 * q], acc[p][q]);
            __syncthreads();
        }
        for (int p = 0; p < 4; ++p)
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + ty + 16 * p, j = j0 + tx + 16 * q;
                if (i >= I || j >= J) continue;
                const int64_t at = KIND == kWgrad
                                       ? (int64_t{e} * a.n + i) * a.k + j
                                       : (int64_t{lo} + i) * a.out_ld + j;
                float v = acc[p][q];
                if (a.out_fp32) {
                    float *o = static_cast<float *>(a.out) + at;
                    *o = KIND == kWgrad && a.accumulate ? *o + v : v;
                } else {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + at;
                    if (KIND == kWgrad && a.accumulate) v += __bfloat162float(*o);
                    *o = __float2bfloat16_rn(v);
                }
            }
    }
}

}  // namespace

cudaError_t launch_grouped_gemm(const GroupedArgs &a, cudaStream_t s) {
    const int J = a.kind == kForward ? a.n : a.k;
    const int64_t I = a.kind == kWgrad ? a.n : a.rows;
    const dim3 grid((J + kTile - 1) / kTile,
                    static_cast<unsigned>(min((I + kTile - 1) / kTile, int64_t{1024})),
                    a.num_experts);
    switch (a.kind) {
        case kForward:
            return launch_ex(grouped_gemm_simple_kernel<kForward>, grid, dim3(256), 0, s, 1,
                             a.programmatic, a);
        case kDgrad:
            return launch_ex(grouped_gemm_simple_kernel<kDgrad>, grid, dim3(256), 0, s, 1,
                             a.programmatic, a);
        default:
            return launch_ex(grouped_gemm_simple_kernel<kWgrad>, grid, dim3(256), 0, s, 1,
                             a.programmatic, a);
    }
}

}  // namespace mf
