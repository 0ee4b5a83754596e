// The tokens' rows into expert order and back, weighted, and the gradients of the way
// back.  With m(t, j) the row of slot j of token t and w(t, j) its routing weight,
//
//   dispatch   out[m(t, j)] = w(t, j) x[t]
//   combine    out[t] = sum_j w(t, j) rows[m(t, j)]             FP32, ascending j
//   backward   d_rows[m(t, j)] = w(t, j) dy[t],   d_w(t, j) = <rows[m(t, j)], dy[t]>
//
// All are bound by the rows' bytes: every row is read or written once, and the token's
// row once for all its slots, by the gradients once for every eight slots (GB300: 8000 x 8
// rows of 7168 154 us into order, 151 back, 290 for both gradients, 6.7 - 6.8 TB/s, the
// copy's rate; both gradients of 2000 x 8, 16 and 32 rows of 4096 46, 88 and 174 us).  A slot without a row (m outside the
// rows) moves nothing, and its weight is not used.
#include "experts.h"
#include "rows.cuh"

namespace mf {
namespace {

constexpr int kAhead = 4;      // slots whose rows are loaded before the first is used
constexpr int kThreads = 128;  // of a CTA

// Columns that a thread takes at a time: 16 bytes of the wider type, so that neighbouring
// threads' accesses touch whole 32-byte sectors (of 8 FP32 values, two accesses touch half
// of each: 1031 x 5 rows of 2872 took 19.2 us into order, 517 x 6 of 2056 14.8 for the
// gradients; 12.4 and 11.3 so).
template <bool A_FP32, bool B_FP32>
constexpr int kColumns = A_FP32 || B_FP32 ? 4 : 8;

template <bool FP32, int N>
struct Columns {
    static_assert(N == 4 || (N == 8 && !FP32), "up to 16 bytes");
    uint32_t v[FP32 ? N : N / 2];

    __device__ void load(const void *rows, int64_t at, bool read) {
        const uint8_t *p = static_cast<const uint8_t *>(rows) + at * (FP32 ? 4 : 2);
        if constexpr (FP32 || N == 8) {
            const uint4 q = ld_nc_na_16_if(p, read);
            v[0] = q.x;
            v[1] = q.y;
            v[2] = q.z;
            v[3] = q.w;
        } else {
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\t"
                "@p ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n\t}"
                : "=&r"(v[0]), "=&r"(v[1])
                : "l"(p), "r"(uint32_t{read}));
        }
    }
    __device__ void get(float (&f)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = FP32 ? __uint_as_float(v[FP32 ? i : 0])
                        : i % 2 ? bf16_hi(v[FP32 ? 0 : i / 2]) : bf16_lo(v[FP32 ? 0 : i / 2]);
    }
    // Rounded once, written once (streaming).
    static __device__ void store(void *rows, int64_t at, const float (&f)[N]) {
        if constexpr (FP32) {
            st_cs_16(static_cast<float *>(rows) + at,
                     make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                __float_as_uint(f[3])));
        } else if constexpr (N == 8) {
            st_cs_16(static_cast<__nv_bfloat16 *>(rows) + at, pack8_rn(f));
        } else {
            asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(
                             static_cast<__nv_bfloat16 *>(rows) + at),
                         "r"(pack2_rn(f[0], f[1])), "r"(pack2_rn(f[2], f[3]))
                         : "memory");
        }
    }
};

// A thread takes N columns of a token for all its slots.
template <bool IN_FP32, bool OUT_FP32>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(CombineArgs a) {
    constexpr int N = kColumns<IN_FP32, OUT_FP32>;
    pdl_wait();
    const int chunks = a.hidden / N;
    const int64_t i = blockIdx.x * int64_t{kThreads} + threadIdx.x;
    if (i >= a.num_tokens * chunks) return;
    const int64_t t = i / chunks;
    const int c = static_cast<int>(i - t * chunks) * N;
    const int32_t *idx = a.idx + t * a.top_k;
    Columns<IN_FP32, N> q;
    q.load(a.token_rows, t * a.token_ld + c, true);
    float x[N];
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
            float y[N];
#pragma unroll
            for (int u = 0; u < N; ++u) y[u] = w[j] * x[u];
            Columns<OUT_FP32, N>::store(a.out_rows, row[j] * a.out_ld + c, y);
        }
    }
}

template <bool IN_FP32, bool OUT_FP32>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a) {
    constexpr int N = kColumns<IN_FP32, OUT_FP32>;
    pdl_wait();
    const int chunks = a.hidden / N;
    const int64_t i = blockIdx.x * int64_t{kThreads} + threadIdx.x;
    if (i >= a.num_tokens * chunks) return;
    const int64_t t = i / chunks;
    const int c = static_cast<int>(i - t * chunks) * N;
    const int32_t *idx = a.idx + t * a.top_k;
    float acc[N] = {};
    for (int j0 = 0; j0 < a.top_k; j0 += kAhead) {
        Columns<IN_FP32, N> q[kAhead];
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
            float f[N];
            q[j].get(f);
#pragma unroll
            for (int u = 0; u < N; ++u) acc[u] = fmaf(w[j], f[u], acc[u]);
        }
    }
    Columns<OUT_FP32, N>::store(a.out_rows, t * a.out_ld + c, acc);
}

// Sums of N values (a power of two) over the warp: value i ends in the 32 / N lanes from
// 32 / N i on.  Each step halves the values a lane holds and exchanges the other half with
// the lane across.
template <int N>
__device__ __forceinline__ float warp_sums(const float (&v)[N], int across = 16) {
    if constexpr (N == 1) {
        float s = v[0];
        for (; across > 0; across /= 2) s += __shfl_xor_sync(0xffffffffu, s, across);
        return s;
    } else {
        const bool up = threadIdx.x & across;
        float half[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float give = up ? v[i] : v[i + N / 2];
            half[i] = (up ? v[i + N / 2] : v[i]) + __shfl_xor_sync(0xffffffffu, give, across);
        }
        return warp_sums(half, across / 2);
    }
}

// A token's gradients by a team of TEAM threads (several teams to a CTA where a row is
// short): each takes every TEAM-th chunk of N columns, for kSlots slots at a time; the dot
// products are added up over the warp and then over the team's warps, in one order
// always.  WRITE: d_rows are wanted beside d_w.
template <bool DY_FP32, bool ROWS_FP32, int TEAM, int kSlots, bool WRITE>
__global__ void __launch_bounds__(TEAM < 128 ? 128 : TEAM) combine_backward_kernel(CombineArgs a) {
    constexpr int kCta = TEAM < 128 ? 128 : TEAM;
    constexpr int kLanes = 32 / kSlots;  // that hold a slot's sum
    constexpr int N = kColumns<DY_FP32, ROWS_FP32>;
    __shared__ float sums[kCta / 32][kSlots];
    pdl_wait();
    const int team = threadIdx.x / TEAM, member = threadIdx.x % TEAM;
    const int64_t t = blockIdx.x * int64_t{kCta / TEAM} + team;
    const bool live = t < a.num_tokens;
    const int chunks = live ? a.hidden / N : 0;
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
            Columns<DY_FP32, N> d;
            d.load(a.token_rows, t * a.token_ld + c * N, true);
            Columns<ROWS_FP32, N> q[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                q[j].load(a.rows, row[j] * a.ld + c * N, row[j] >= 0);
            float dy[N];
            d.get(dy);
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                float f[N];
                q[j].get(f);
                // two chains, so that a chunk's products are not one long one
                float even = f[0] * dy[0], odd = f[1] * dy[1];
#pragma unroll
                for (int u = 2; u < N; u += 2) {
                    even = fmaf(f[u], dy[u], even);
                    odd = fmaf(f[u + 1], dy[u + 1], odd);
                }
                if (row[j] >= 0) {
                    dot[j] += even + odd;
                    if (WRITE) {
                        float y[N];
#pragma unroll
                        for (int u = 0; u < N; ++u) y[u] = w[j] * dy[u];
                        Columns<ROWS_FP32, N>::store(a.out_rows, row[j] * a.out_ld + c * N, y);
                    }
                }
            }
        }
        const float s = warp_sums(dot);
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const int slot = lane / kLanes;
        float total = s;
        if (TEAM > 32) {
            if (lane % kLanes == 0) sums[warp][slot] = s;
            __syncthreads();
            total = 0.f;
            if (member < 32)
                for (int i = 0; i < TEAM / 32; ++i) total += sums[warp + i][slot];
            __syncthreads();  // before the next slots' sums
        }
        if (live && member < 32 && lane % kLanes == 0 && j0 + slot < a.top_k) {
            const int64_t at = t * a.top_k + j0 + slot;
            if (a.grad_weights_fp32)
                static_cast<float *>(a.grad_weights)[at] = total;
            else
                static_cast<__nv_bfloat16 *>(a.grad_weights)[at] = __float2bfloat16_rn(total);
        }
    }
}

template <bool DY_FP32, bool ROWS_FP32, int TEAM, int SLOTS>
cudaError_t launch_backward(const CombineArgs &a, cudaStream_t s) {
    constexpr int kCta = TEAM < 128 ? 128 : TEAM;
    const dim3 grid(static_cast<unsigned>((a.num_tokens + kCta / TEAM - 1) / (kCta / TEAM)));
    if (a.out_rows)
        return launch_ex(combine_backward_kernel<DY_FP32, ROWS_FP32, TEAM, SLOTS, true>, grid,
                         dim3(kCta), 0, s, 1, a.programmatic, a);
    return launch_ex(combine_backward_kernel<DY_FP32, ROWS_FP32, TEAM, SLOTS, false>, grid,
                     dim3(kCta), 0, s, 1, a.programmatic, a);
}

// How many threads take a token.  A warp where rows are short and tokens many, up to 192
// chunks (8000 x 8 rows, a warp against 128 threads: 64 chunks 25.4 and 40.5 us, 128 47.3 and
// 50.4, 192 68.6 and 72.7, 256 89.7 and 87.2; 8000 x 4 rows 14.0 and 18.2, 25.0 and 24.9, 36.3
// and 36.1, 47.2 and 45.6).  Of fewer tokens a warp each does not fill the SMs (1000 x 8 rows,
// 192 chunks: 13.2 and 12.1; 153 x 8: 8.6 and 4.6): the rule has them wrong by that.  512
// threads where there is a token to an SM at most (152 x 8 rows, 264 chunks 4.5 us and 6.0 with
// 128 threads, 896 chunks 8.8 and 11.9; 153 x 8 rows 6.8 and 6.0, 11.9 and 12.0).
template <bool DY_FP32, bool ROWS_FP32, int SLOTS>
cudaError_t launch_team(const CombineArgs &a, cudaStream_t s) {
    const int chunks = a.hidden / kColumns<DY_FP32, ROWS_FP32>;
    if (chunks <= 192 && a.num_tokens > a.num_sms)
        return launch_backward<DY_FP32, ROWS_FP32, 32, SLOTS>(a, s);
    if (chunks > 256 && a.num_tokens <= a.num_sms)
        return launch_backward<DY_FP32, ROWS_FP32, 512, SLOTS>(a, s);
    return launch_backward<DY_FP32, ROWS_FP32, 128, SLOTS>(a, s);
}

template <bool DY_FP32, bool ROWS_FP32>
cudaError_t launch_slots(const CombineArgs &a, cudaStream_t s) {
    return a.top_k <= 4 ? launch_team<DY_FP32, ROWS_FP32, 4>(a, s)
                        : launch_team<DY_FP32, ROWS_FP32, 8>(a, s);
}

dim3 chunk_grid(const CombineArgs &a) {
    const int columns = a.token_fp32 || a.rows_fp32 ? 4 : 8;
    return dim3(
        static_cast<unsigned>((a.num_tokens * (a.hidden / columns) + kThreads - 1) / kThreads));
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
        return a.rows_fp32 ? launch_slots<true, true>(a, s) : launch_slots<true, false>(a, s);
    return a.rows_fp32 ? launch_slots<false, true>(a, s) : launch_slots<false, false>(a, s);
}

}  // namespace mf
