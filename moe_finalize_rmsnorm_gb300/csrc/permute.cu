// Permutation by expert and the gradient of the gather it defines.
#include "experts.cuh"
#include "experts.h"

namespace mf {
namespace {

// Permutation: a stable counting sort.
//
// Latency bound: 12 bytes a slot move in under a microsecond even for 262144
// slots, so what counts is the number of dependent steps.  Up to kOneCta slots one
// CTA does everything (256 slots 2.6 us; 2400 slots 6.1 against 7.7 us for the two
// launches, 4000 7.7 either way, 8000 12.1 against 7.7).  Beyond, two launches: a cluster
// counts the slots chunk by chunk and turns the counts into each chunk's first row
// per expert, and a CTA for every chunk places its slots.  The first rows need no
// workspace: a chunk is at least as long as there are experts, so they lie in its
// own part of the slot-to-row map until its CTA has read them and writes the map
// itself.

constexpr int kPermuteThreads = 1024;
constexpr int kPermuteWarps = kPermuteThreads / 32;
constexpr int kOneCta = 4096;
constexpr int kChunk = 1024;      // slots of a chunk, at least (the last up to twice as many)
constexpr int kMaxChunks = 152;
// CTAs of the cluster that counts: 8, from kManySlots on 16, the largest there is
// (64000 slots 12.0 against 13.3 us, 262144 slots 13.8 against 11.7 us).
constexpr int kCountCtas = 8;
constexpr int64_t kManySlots = 131072;
static_assert(kChunk >= kMaxExperts, "a chunk's first rows lie in its part of the map");

// Expert of a slot, -1 when it has none among [0, E).
__device__ __forceinline__ int slot_expert(int word, int packed, int num_experts) {
    const unsigned id = packed ? static_cast<unsigned>(word) >> 16 : static_cast<unsigned>(word);
    return id < static_cast<unsigned>(num_experts) ? static_cast<int>(id) : -1;
}

// Exclusive sum over the CTA's 1024 threads; `total` is the sum of all.
__device__ __forceinline__ int block_scan(int v, int32_t *scratch, int &total) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int sum = v;
    for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    int w = scratch[lane];
    for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return sum - v + (warp ? before : 0);
}

// Hand the slots [begin, end) of a warp their rows, in slot order.  next[e] is the
// row of the warp's next slot with expert e (plus base[e]); match_any gives a slot
// its rank among the warp's 32.
__device__ __forceinline__ void place(const PermuteArgs &a, int64_t begin, int64_t end,
                                      int32_t *next, const int32_t *base) {
    const int lane = threadIdx.x % 32;
    for (int64_t s = begin; s < end; s += 32) {
        const bool in = s + lane < end;
        const int e = in ? slot_expert(a.ids[s + lane], a.packed, a.num_experts) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int first = e >= 0 ? next[e] : 0;
        __syncwarp();
        if (e >= 0) {
            const int row = base[e] + first + rank;
            a.slot_to_row[s + lane] = row;
            a.row_to_token[row] =
                static_cast<int32_t>(static_cast<uint32_t>(s + lane) / static_cast<uint32_t>(a.top_k));
            if (rank == 0) next[e] = first + __popc(same);
        } else if (in) {
            a.slot_to_row[s + lane] = -1;
        }
        __syncwarp();
    }
}

// The slots [begin, end) of this warp counted into mine[e].
__device__ __forceinline__ void count(const PermuteArgs &a, int64_t begin, int64_t end,
                                      int32_t *mine) {
    for (int64_t s = begin + threadIdx.x % 32; s < end; s += 32) {
        const int e = slot_expert(a.ids[s], a.packed, a.num_experts);
        if (e >= 0) atomicAdd(mine + e, 1);
    }
}

// counts[w][e] of `warps` warps to each warp's first position; returns the sums of
// this thread's expert.
__device__ __forceinline__ int warp_prefix(int32_t *counts, int warps, int num_experts) {
    int sum = 0;
    const int e = threadIdx.x;
    if (e < num_experts)
        for (int w = 0; w < warps; ++w) {
            const int c = counts[w * num_experts + e];
            counts[w * num_experts + e] = sum;
            sum += c;
        }
    return sum;
}

__global__ void __launch_bounds__(kPermuteThreads) permute_one_cta_kernel(PermuteArgs a, int warps) {
    extern __shared__ int32_t counts[];  // [warps][E]
    __shared__ int32_t base[kMaxExperts];
    __shared__ int32_t scratch[32];
    const int warp = threadIdx.x / 32;
    const int E = a.num_experts;
    for (int i = threadIdx.x; i < warps * E; i += kPermuteThreads) counts[i] = 0;
    __syncthreads();
    pdl_wait();
    const int64_t per_warp = (a.slots + 32 * warps - 1) / (32 * warps) * 32;
    const int64_t begin = min(per_warp * warp, a.slots), end = min(begin + per_warp, a.slots);
    if (warp < warps) count(a, begin, end, counts + warp * E);
    __syncthreads();
    const int sum = warp_prefix(counts, warps, E);
    int total;
    const int offset = block_scan(sum, scratch, total);
    if (threadIdx.x < E) {
        base[threadIdx.x] = offset;
        a.offsets[threadIdx.x] = offset;
    }
    if (threadIdx.x == 0) a.offsets[E] = total;
    __syncthreads();
    if (warp < warps) place(a, begin, end, counts + warp * E, base);
    for (int64_t r = total + threadIdx.x; r < a.slots; r += kPermuteThreads) a.row_to_token[r] = -1;
}

// Slots [begin, end) of chunk c: equal chunks, the last with the remainder.
__device__ __forceinline__ void chunk_slots(const PermuteArgs &a, int c, int chunks, int64_t &begin,
                                            int64_t &end) {
    const int64_t each = a.slots / chunks;
    begin = c * each;
    end = c + 1 == chunks ? a.slots : begin + each;
}

// Every chunk's first row per expert.  Each CTA of the cluster counts a run of
// chunks; the CTAs read each other's sums and scan them all over the experts.
__global__ void __launch_bounds__(kPermuteThreads) permute_count_kernel(PermuteArgs a, int chunks,
                                                                        int ctas) {
    extern __shared__ int32_t counts[];  // [chunks of the CTA][E]
    __shared__ int32_t sums[kMaxExperts];
    __shared__ int32_t scratch[32];
    const int rank = static_cast<int>(cluster_ctarank());
    const int E = a.num_experts;
    const int c0 = chunks * rank / ctas, c1 = chunks * (rank + 1) / ctas;
    for (int i = threadIdx.x; i < (c1 - c0) * E; i += kPermuteThreads) counts[i] = 0;
    __syncthreads();
    pdl_wait();
    const uint32_t each = static_cast<uint32_t>(a.slots / chunks);  // as chunk_slots
    const uint32_t begin = each * c0;
    const uint32_t end = c1 == chunks ? static_cast<uint32_t>(a.slots) : each * c1;
    constexpr int kLoads = 8;  // in flight
    for (uint32_t s0 = begin + threadIdx.x; s0 < end; s0 += kLoads * kPermuteThreads) {
        int word[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (s0 + i * kPermuteThreads < end) word[i] = __ldg(a.ids + s0 + i * kPermuteThreads);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t s = s0 + i * kPermuteThreads;
            if (s >= end) break;
            const int e = slot_expert(word[i], a.packed, E);
            const int c = min(static_cast<int>(s / each), chunks - 1);
            if (e >= 0) atomicAdd(counts + (c - c0) * E + e, 1);
        }
    }
    __syncthreads();
    const int e = threadIdx.x;
    int sum = 0;
    if (e < E)
        for (int c = 0; c < c1 - c0; ++c) sum += counts[c * E + e];
    sums[e] = sum;
    __syncthreads();
    cluster_barrier();
    int before = 0, all = 0;
    if (e < E)
#pragma unroll 8
        for (int r = 0; r < ctas; ++r) {
            const int v = __float_as_int(ld_dsmem_f32(smem_u32(sums + e), r));
            before += r < rank ? v : 0;
            all += v;
        }
    int total;
    const int offset = block_scan(all, scratch, total);
    if (e < E) {
        int row = offset + before;
        for (int c = c0; c < c1; ++c) {
            a.slot_to_row[a.slots / chunks * c + e] = row;
            row += counts[(c - c0) * E + e];
        }
        if (rank == 0) a.offsets[e] = offset;
    }
    if (rank == 0 && e == 0) a.offsets[E] = total;
    __syncthreads();
    cluster_barrier_exit();  // the sums are read
}

__global__ void __launch_bounds__(kPermuteThreads) permute_place_kernel(PermuteArgs a) {
    extern __shared__ int32_t counts[];  // [warps][E]
    __shared__ int32_t base[kMaxExperts];
    const int warp = threadIdx.x / 32;
    const int E = a.num_experts;
    for (int i = threadIdx.x; i < kPermuteWarps * E; i += kPermuteThreads) counts[i] = 0;
    __syncthreads();
    pdl_wait();
    int64_t begin, end;
    chunk_slots(a, blockIdx.x, gridDim.x, begin, end);
    if (threadIdx.x < E) base[threadIdx.x] = a.slot_to_row[begin + threadIdx.x];
    const int64_t per_warp = (end - begin + kPermuteThreads - 1) / kPermuteThreads * 32;
    const int64_t b = min(begin + per_warp * warp, end), e = min(b + per_warp, end);
    count(a, b, e, counts + warp * E);
    __syncthreads();
    (void)warp_prefix(counts, kPermuteWarps, E);
    __syncthreads();
    place(a, b, e, counts + warp * E, base);
    const int total = a.offsets[E];
    for (int64_t r = total + blockIdx.x * int64_t{kPermuteThreads} + threadIdx.x; r < a.slots;
         r += int64_t{gridDim.x} * kPermuteThreads)
        a.row_to_token[r] = -1;
}

// out[t, :] = sum_j rows[idx[t, j], :], FP32 in ascending j: bound by the rows'
// bytes.  A thread takes 16 bytes of a row (32 of an FP32 row), and loads the rows
// of kRowsAhead slots before it adds the first.  8000 x 8 rows of 7168: 149.4 us, 6.91
// TB/s, the copy's rate (two ahead 153, eight 164; 256 threads a CTA 151).
constexpr int kRowsAhead = 4;
constexpr int kSumThreads = 128;

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

template <bool IN_FP32, bool OUT_FP32>
__global__ void __launch_bounds__(kSumThreads) permuted_row_sum_kernel(RowSumArgs a) {
    pdl_wait();
    const int chunks = a.hidden / 8;
    const int64_t i = blockIdx.x * int64_t{kSumThreads} + threadIdx.x;
    if (i >= a.num_tokens * chunks) return;
    const int64_t t = i / chunks;
    const int c = static_cast<int>(i - t * chunks) * 8;
    const int32_t *idx = a.idx + t * a.top_k;
    float acc[8] = {};
    for (int j0 = 0; j0 < a.top_k; j0 += kRowsAhead) {
        Chunk8<IN_FP32> q[kRowsAhead];
#pragma unroll
        for (int j = 0; j < kRowsAhead; ++j) {
            const int r = j0 + j < a.top_k ? __ldg(idx + j0 + j) : -1;
            q[j].load(a.rows, r * a.ld + c, r >= 0 && r < a.num_rows);
        }
#pragma unroll
        for (int j = 0; j < kRowsAhead; ++j) {
            float f[8];
            q[j].get(f);
#pragma unroll
            for (int u = 0; u < 8; ++u) acc[u] += f[u];
        }
    }
    const int64_t at = t * a.hidden + c;
    if (OUT_FP32) {
        float *o = static_cast<float *>(a.out) + at;
        st_cs_16(o, make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]),
                               __float_as_uint(acc[2]), __float_as_uint(acc[3])));
        st_cs_16(o + 4, make_uint4(__float_as_uint(acc[4]), __float_as_uint(acc[5]),
                                   __float_as_uint(acc[6]), __float_as_uint(acc[7])));
    } else {
        st_cs_16(static_cast<__nv_bfloat16 *>(a.out) + at, pack8_rn(acc));
    }
}

}  // namespace

cudaError_t prepare_permute_kernels(bool *wide_clusters) {
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const int bytes = kPermuteWarps * kMaxExperts * 4;
    cudaError_t e = cudaFuncSetAttribute(permute_one_cta_kernel, attr, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(permute_count_kernel,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(permute_count_kernel, attr,
                                 (kMaxChunks + kCountCtas - 1) / kCountCtas * kMaxExperts * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(permute_place_kernel, attr, bytes);
    if (e != cudaSuccess) return e;
    // clusters of 16 are not portable: whether this device has room for one
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute wide = {};
    wide.id = cudaLaunchAttributeClusterDimension;
    wide.val.clusterDim.x = 2 * kCountCtas;
    wide.val.clusterDim.y = wide.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * kCountCtas);
    cfg.blockDim = dim3(kPermuteThreads);
    cfg.dynamicSmemBytes = (kMaxChunks + kCountCtas - 1) / kCountCtas * kMaxExperts * 4;
    cfg.attrs = &wide;
    cfg.numAttrs = 1;
    int clusters = 0;
    *wide_clusters =
        cudaOccupancyMaxActiveClusters(&clusters, permute_count_kernel, &cfg) == cudaSuccess &&
        clusters > 0;
    (void)cudaGetLastError();
    return cudaSuccess;
}

cudaError_t launch_expert_permutation(const PermuteArgs &a, cudaStream_t s) {
    const dim3 block(kPermuteThreads);
    if (a.slots <= kOneCta) {
        const int warps =
            static_cast<int>(min(max((a.slots + 31) / 32, int64_t{1}), int64_t{kPermuteWarps}));
        return launch_ex(permute_one_cta_kernel, dim3(1), block,
                         sizeof(int32_t) * warps * a.num_experts, s, 1, a.programmatic, a,
                         warps);
    }
    const int chunks = static_cast<int>(min(a.slots / kChunk, int64_t{kMaxChunks}));
    const int ctas = a.slots < kManySlots || !a.wide_clusters ? kCountCtas : 2 * kCountCtas;
    cudaError_t e = launch_ex(permute_count_kernel, dim3(ctas), block,
                              sizeof(int32_t) * ((chunks + ctas - 1) / ctas) * a.num_experts, s,
                              ctas, a.programmatic, a, chunks, ctas);
    if (e == cudaSuccess)
        e = launch_ex(permute_place_kernel, dim3(chunks), block,
                      sizeof(int32_t) * kPermuteWarps * a.num_experts, s, 1, a.programmatic, a);
    return e;
}

cudaError_t launch_permuted_row_sum(const RowSumArgs &a, cudaStream_t s) {
    const int64_t threads = a.num_tokens * (a.hidden / 8);
    const dim3 grid(static_cast<unsigned>((threads + kSumThreads - 1) / kSumThreads)),
        block(kSumThreads);
    if (a.rows_fp32 && a.out_fp32)
        return launch_ex(permuted_row_sum_kernel<true, true>, grid, block, 0, s, 1,
                         a.programmatic, a);
    if (a.rows_fp32)
        return launch_ex(permuted_row_sum_kernel<true, false>, grid, block, 0, s, 1,
                         a.programmatic, a);
    if (a.out_fp32)
        return launch_ex(permuted_row_sum_kernel<false, true>, grid, block, 0, s, 1,
                         a.programmatic, a);
    return launch_ex(permuted_row_sum_kernel<false, false>, grid, block, 0, s, 1,
                     a.programmatic, a);
}

}  // namespace mf
