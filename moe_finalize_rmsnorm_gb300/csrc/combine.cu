// The tokens' rows into expert order and back, weighted, and the gradients of the way
// back.  With m(t, j) the row of slot j of token t and w(t, j) its routing weight,
//
//   dispatch   out[m(t, j)] = w(t, j) x[t]
//   combine    out[t] = sum_j w(t, j) rows[m(t, j)]             FP32, ascending j
//   backward   d_rows[m(t, j)] = w(t, j) dy[t],   d_w(t, j) = <rows[m(t, j)], dy[t]>
//
// All are bound by the rows' bytes: every row is read or written once, and the token's
// row once for all its slots.  A slot without a row (m outside the rows) moves nothing,
// and its weight is not used.
#include "experts.h"
#include "rows.cuh"

namespace mf {
namespace {

constexpr int kAhead = 4;      // slots whose rows are loaded before the first is used
constexpr int kThreads = 128;  // of a CTA

// A thread takes 8 columns of a token for all its slots.
template <bool IN_FP32, bool OUT_FP32>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(CombineArgs a) {
    pdl_wait();
    const int chunks = a.hidden / 8;
    const int64_t i = blockIdx.x * int64_t{kThreads} + threadIdx.x;
    if (i >= a.num_tokens * chunks) return;
    const int64_t t = i / chunks;
    const int c = static_cast<int>(i - t * chunks) * 8;
    const int32_t *idx = a.idx + t * a.top_k;
    Chunk8<IN_FP32> q;
    q.load(a.token_rows, t * a.token_ld + c, true);
    float x[8];
    q.get(x);
    for (int j0 = 0; j0 < a.top_k; j0 += kAhead) {
        int row[kAhead];
        float w[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) row[j] = j0 + j < a.top_k ? __ldg(idx + j0 + j) : -1;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (row[j] >= a.num_rows) row[j] = -1;
            w[j] = row[j] >= 0
                       ? routing_weight(a.weights, a.weight_kind, t * a.top_k + j0 + j)
                       : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (row[j] < 0) continue;
            float y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) y[u] = w[j] * x[u];
            store8<OUT_FP32>(a.out_rows, row[j] * a.out_ld + c, y);
        }
    }
}

template <bool IN_FP32, bool OUT_FP32>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a) {
    pdl_wait();
    const int chunks = a.hidden / 8;
    const int64_t i = blockIdx.x * int64_t{kThreads} + threadIdx.x;
    if (i >= a.num_tokens * chunks) return;
    const int64_t t = i / chunks;
    const int c = static_cast<int>(i - t * chunks) * 8;
    const int32_t *idx = a.idx + t * a.top_k;
    float acc[8] = {};
    for (int j0 = 0; j0 < a.top_k; j0 += kAhead) {
        Chunk8<IN_FP32> q[kAhead];
        float w[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int r = j0 + j < a.top_k ? __ldg(idx + j0 + j) : -1;
            const bool valid = r >= 0 && r < a.num_rows;
            q[j].load(a.rows, r * a.ld + c, valid);
            w[j] = valid ? routing_weight(a.weights, a.weight_kind, t * a.top_k + j0 + j) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            float f[8];
            q[j].get(f);
#pragma unroll
            for (int u = 0; u < 8; ++u) acc[u] = fmaf(w[j], f[u], acc[u]);
        }
    }
    store8<OUT_FP32>(a.out_rows, t * a.out_ld + c, acc);
}

// Sums of eight values over the warp: lane 4 i (of every four) ends with value i.
__device__ __forceinline__ float warp_sum8(const float (&v)[8]) {
    const int lane = threadIdx.x % 32;
    float a[4], b[2];
    // halve the values held, exchanging the other half with the lane across
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        const float give = up ? v[i] : v[i + 4];
        a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        const float give = up ? a[i] : a[i + 2];
        b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, give, 8);
    }
    const bool up = lane & 4;
    const float give = up ? b[0] : b[1];
    float s = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, give, 4);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    return s + __shfl_xor_sync(0xffffffffu, s, 1);
}

// A token's gradients by a team of TEAM threads (several teams to a CTA where a row is
// short): each takes every TEAM-th chunk of 8 columns, for 8 slots at a time; the dot
// products are added up over the warp and then over the team's warps, in one order
// always.  WRITE: d_rows are wanted beside d_w.
template <bool DY_FP32, bool ROWS_FP32, int TEAM, bool WRITE>
__global__ void __launch_bounds__(TEAM < 128 ? 128 : TEAM) combine_backward_kernel(CombineArgs a) {
    constexpr int kCta = TEAM < 128 ? 128 : TEAM;
    constexpr int kSlots = 8;
    __shared__ float sums[kCta / 32][kSlots];
    pdl_wait();
    const int team = threadIdx.x / TEAM, member = threadIdx.x % TEAM;
    const int64_t t = blockIdx.x * int64_t{kCta / TEAM} + team;
    const bool live = t < a.num_tokens;
    const int chunks = live ? a.hidden / 8 : 0;
    for (int j0 = 0; j0 < a.top_k; j0 += kSlots) {
        int row[kSlots];
        float w[kSlots], dot[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            row[j] = live && j0 + j < a.top_k ? __ldg(a.idx + t * a.top_k + j0 + j) : -1;
            if (row[j] >= a.num_rows) row[j] = -1;
            w[j] = WRITE && row[j] >= 0
                       ? routing_weight(a.weights, a.weight_kind, t * a.top_k + j0 + j)
                       : 0.f;
            dot[j] = 0.f;
        }
        for (int c = member; c < chunks; c += TEAM) {
            Chunk8<DY_FP32> d;
            d.load(a.token_rows, t * a.token_ld + c * 8, true);
            Chunk8<ROWS_FP32> q[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                q[j].load(a.rows, row[j] * a.ld + c * 8, row[j] >= 0);
            float dy[8];
            d.get(dy);
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                float f[8];
                q[j].get(f);
                // two chains, so that a chunk's eight products are not one long one
                float even = f[0] * dy[0], odd = f[1] * dy[1];
#pragma unroll
                for (int u = 2; u < 8; u += 2) {
                    even = fmaf(f[u], dy[u], even);
                    odd = fmaf(f[u + 1], dy[u + 1], odd);
                }
                if (row[j] >= 0) {
                    dot[j] += even + odd;
                    if (WRITE) {
                        float y[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) y[u] = w[j] * dy[u];
                        store8<ROWS_FP32>(a.out_rows, row[j] * a.out_ld + c * 8, y);
                    }
                }
            }
        }
        const float s = warp_sum8(dot);
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        float total = s;  // of slot lane / 4
        if (TEAM > 32) {
            if (lane % 4 == 0) sums[warp][lane / 4] = s;
            __syncthreads();
            total = 0.f;
            if (member < 32)
                for (int i = 0; i < TEAM / 32; ++i) total += sums[warp + i][lane / 4];
            __syncthreads();  // before the next slots' sums
        }
        if (live && member < 32 && lane % 4 == 0 && j0 + lane / 4 < a.top_k) {
            const int64_t at = t * a.top_k + j0 + lane / 4;
            if (a.grad_weights_fp32)
                static_cast<float *>(a.grad_weights)[at] = total;
            else
                static_cast<__nv_bfloat16 *>(a.grad_weights)[at] = __float2bfloat16_rn(total);
        }
    }
}

template <bool DY_FP32, bool ROWS_FP32, int TEAM>
cudaError_t launch_backward(const CombineArgs &a, cudaStream_t s) {
    constexpr int kCta = TEAM < 128 ? 128 : TEAM;
    const dim3 grid(static_cast<unsigned>((a.num_tokens + kCta / TEAM - 1) / (kCta / TEAM)));
    if (a.out_rows)
        return launch_ex(combine_backward_kernel<DY_FP32, ROWS_FP32, TEAM, true>, grid, dim3(kCta),
                         0, s, 1, a.programmatic, a);
    return launch_ex(combine_backward_kernel<DY_FP32, ROWS_FP32, TEAM, false>, grid, dim3(kCta), 0,
                     s, 1, a.programmatic, a);
}

template <bool DY_FP32, bool ROWS_FP32>
cudaError_t launch_team(const CombineArgs &a, cudaStream_t s) {
    const int chunks = a.hidden / 8;
    if (chunks <= 64) return launch_backward<DY_FP32, ROWS_FP32, 32>(a, s);
    if (a.num_tokens <= 4 * a.num_sms && chunks > 256)
        return launch_backward<DY_FP32, ROWS_FP32, 512>(a, s);
    return launch_backward<DY_FP32, ROWS_FP32, 128>(a, s);
}

dim3 chunk_grid(const CombineArgs &a) {
    return dim3(static_cast<unsigned>((a.num_tokens * (a.hidden / 8) + kThreads - 1) / kThreads));
}

}  // namespace

cudaError_t launch_dispatch(const CombineArgs &a, cudaStream_t s) {
    const auto go = [&](auto kernel) {
        return launch_ex(kernel, chunk_grid(a), dim3(kThreads), 0, s, 1, a.programmatic, a);
    };
    if (a.token_fp32)
        return a.rows_fp32 ? go(dispatch_kernel<true, true>) : go(dispatch_kernel<true, false>);
    return a.rows_fp32 ? go(dispatch_kernel<false, true>) : go(dispatch_kernel<false, false>);
}

cudaError_t launch_combine(const CombineArgs &a, cudaStream_t s) {
    const auto go = [&](auto kernel) {
        return launch_ex(kernel, chunk_grid(a), dim3(kThreads), 0, s, 1, a.programmatic, a);
    };
    if (a.rows_fp32)
        return a.token_fp32 ? go(combine_kernel<true, true>) : go(combine_kernel<true, false>);
    return a.token_fp32 ? go(combine_kernel<false, true>) : go(combine_kernel<false, false>);
}

cudaError_t launch_combine_backward(const CombineArgs &a, cudaStream_t s) {
    if (!a.grad_weights) return launch_dispatch(a, s);  // d_rows alone: the weighted way in
    if (a.token_fp32)
        return a.rows_fp32 ? launch_team<true, true>(a, s) : launch_team<true, false>(a, s);
    return a.rows_fp32 ? launch_team<false, true>(a, s) : launch_team<false, false>(a, s);
}

}  // namespace mf
