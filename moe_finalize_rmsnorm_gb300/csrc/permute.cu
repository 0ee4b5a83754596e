// Permutation by expert and the gradient of the gather it defines.
#include "experts.cuh"
#include "experts.h"

namespace mf {
namespace {

constexpr int kPermuteThreads = 1024;
constexpr int kPermuteWarps = kPermuteThreads / 32;

// Expert of a slot, -1 when it has none among [0, E).
__device__ __forceinline__ int slot_expert(int word, int packed, int num_experts) {
    const unsigned id = packed ? static_cast<unsigned>(word) >> 16 : static_cast<unsigned>(word);
    return id < static_cast<unsigned>(num_experts) ? static_cast<int>(id) : -1;
}

// Stable counting sort by one CTA.  Warp w owns a contiguous run of the slots;
// count[w][e] is its histogram.  A scan over (e, w) turns the counts into each
// warp's next position per expert, and a second pass over the slots hands the
// positions out in slot order (match_any gives a slot its rank among the
// warp's 32).
__global__ void __launch_bounds__(kPermuteThreads) expert_permutation_kernel(PermuteArgs a) {
    extern __shared__ int32_t count[];  // [warps][E]
    __shared__ int32_t total[kMaxExperts + 1];
    pdl_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int E = a.num_experts;
    for (int i = threadIdx.x; i < kPermuteWarps * E; i += kPermuteThreads) count[i] = 0;
    __syncthreads();

    const int64_t per_warp = (a.slots + 32 * kPermuteWarps - 1) / (32 * kPermuteWarps) * 32;
    const int64_t begin = min(per_warp * warp, a.slots);
    const int64_t end = min(begin + per_warp, a.slots);
    int32_t *mine = count + warp * E;
    for (int64_t s = begin; s < end; s += 32) {
        const int e = s + lane < end ? slot_expert(a.ids[s + lane], a.packed, E) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kPermuteThreads) {
        int32_t sum = 0;
        for (int w = 0; w < kPermuteWarps; ++w) {
            const int32_t c = count[w * E + e];
            count[w * E + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int32_t sum = 0;
        for (int e = 0; e < E; ++e) {
            const int32_t c = total[e];
            total[e] = sum;
            sum += c;
        }
        total[E] = sum;
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kPermuteThreads) a.offsets[e] = total[e];
    for (int64_t s = begin; s < end; s += 32) {
        const bool in = s + lane < end;
        const int e = in ? slot_expert(a.ids[s + lane], a.packed, E) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int base = e >= 0 ? mine[e] : 0;
        __syncwarp();
        if (e >= 0) {
            const int row = total[e] + base + rank;
            a.slot_to_row[s + lane] = row;
            a.row_to_token[row] = static_cast<int32_t>((s + lane) / a.top_k);
            if (rank == 0) mine[e] = base + __popc(same);
        } else if (in) {
            a.slot_to_row[s + lane] = -1;
        }
        __syncwarp();
    }
    for (int64_t r = total[E] + threadIdx.x; r < a.slots; r += kPermuteThreads)
        a.row_to_token[r] = -1;
}

// out[t, :] = sum_j rows[idx[t, j], :], FP32 in ascending j, one thread per
// eight columns of a token.
template <typename In, typename Out>
__global__ void __launch_bounds__(256) permuted_row_sum_kernel(RowSumArgs a) {
    pdl_wait();
    const int chunks = a.hidden / 8;
    const int64_t i = blockIdx.x * int64_t{256} + threadIdx.x;
    if (i >= a.num_tokens * chunks) return;
    const int64_t t = i / chunks;
    const int c = static_cast<int>(i % chunks) * 8;
    float acc[8] = {};
    for (int j = 0; j < a.top_k; ++j) {
        const int64_t r = a.idx[t * a.top_k + j];
        if (r < 0 || r >= a.num_rows) continue;
        const In *p = static_cast<const In *>(a.rows) + r * a.ld + c;
        for (int u = 0; u < 8; ++u) acc[u] += static_cast<float>(p[u]);
    }
    Out *o = static_cast<Out *>(a.out) + t * a.hidden + c;
    for (int u = 0; u < 8; ++u) o[u] = static_cast<Out>(acc[u]);
}

}  // namespace

cudaError_t prepare_permute_kernels() {
    return cudaFuncSetAttribute(expert_permutation_kernel,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kPermuteWarps * kMaxExperts * 4);
}

cudaError_t launch_expert_permutation(const PermuteArgs &a, cudaStream_t s) {
    return launch_ex(expert_permutation_kernel, dim3(1), dim3(kPermuteThreads),
                     sizeof(int32_t) * kPermuteWarps * a.num_experts, s, 1, a.programmatic, a);
}

cudaError_t launch_permuted_row_sum(const RowSumArgs &a, cudaStream_t s) {
    const int64_t threads = a.num_tokens * (a.hidden / 8);
    const dim3 grid(static_cast<unsigned>((threads + 255) / 256)), block(256);
    if (a.rows_fp32 && a.out_fp32)
        return launch_ex(permuted_row_sum_kernel<float, float>, grid, block, 0, s, 1,
                         a.programmatic, a);
    if (a.rows_fp32)
        return launch_ex(permuted_row_sum_kernel<float, __nv_bfloat16>, grid, block, 0, s, 1,
                         a.programmatic, a);
    if (a.out_fp32)
        return launch_ex(permuted_row_sum_kernel<__nv_bfloat16, float>, grid, block, 0, s, 1,
                         a.programmatic, a);
    return launch_ex(permuted_row_sum_kernel<__nv_bfloat16, __nv_bfloat16>, grid, block, 0, s, 1,
                     a.programmatic, a);
}

}  // namespace mf
