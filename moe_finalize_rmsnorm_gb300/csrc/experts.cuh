// Device helpers shared by the expert-layer kernels.
#pragma once

#include "common.cuh"

namespace mf {

// The experts' rows and the numbers of their passes (of up to `per_pass` rows):
// lo[e] is the first row, lo[num_experts] the end; passes[e] counts the passes of the
// experts before e.  Called by the whole CTA, of which `THREADS` threads take a run of
// experts each; `scratch` holds an int per warp of theirs.  Returns the passes of all
// experts; the tables are complete after the caller's next barrier.
//
// The offsets are device data that the host cannot check, so they are brought into
// [0, rows], and offsets that do not ascend give no passes at all: experts that overlap
// could have more of them than 32 bits count, and an item number that wraps around would
// reach outside the buffers.
template <int THREADS>
__device__ __forceinline__ int scan_experts(const int32_t *offsets, int num_experts, int rows,
                                            int per_pass, int *lo, int *passes, int *scratch) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per = (num_experts + THREADS - 1) / THREADS;
    const int first = min(static_cast<int>(threadIdx.x) * per, num_experts);
    const int last = min(first + per, num_experts);
    int sum = 0;
    bool ascend = true;
    for (int e = first; e < last; ++e) {
        int l = 0, h = rows;  // without offsets one expert has every row
        if (offsets) {
            l = min(max(__ldg(offsets + e), 0), rows);
            h = min(max(__ldg(offsets + e + 1), 0), rows);
        }
        ascend = ascend && l <= h;
        lo[e] = l;
        if (e + 1 == num_experts) lo[e + 1] = h;
        passes[e] = sum;
        if (ascend) sum += (h - l + per_pass - 1) / per_pass;  // a run of up to `rows` rows
    }
    int before = sum;
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31 && warp < THREADS / 32) scratch[warp] = before;
    before -= sum;
    if (__syncthreads_or(!ascend)) return 0;
    int total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    for (int e = first; e < last; ++e) passes[e] += before;
    if (threadIdx.x == 0) passes[num_experts] = total;
    return total;
}

// The expert of a pass: the last whose passes start at or before it.  `step` is the
// largest power of two up to the number of experts.
__device__ __forceinline__ int expert_of_pass(const int *passes, int num_experts, int step,
                                              int pass) {
    int e = 0;
    for (; step > 0; step /= 2)
        if (e + step < num_experts && passes[e + step] <= pass) e += step;
    return e;
}

// mbar_wait of common.cuh for waits that are long and many (a persistent kernel's
// roles wait for each other all the time): each try may suspend the thread for up to
// a millisecond, so that a waiting warp issues next to nothing.  CLUSTER: the arrivals
// may come from the other CTA of a pair, so the wait acquires at cluster scope (no
// difference in time).
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    const auto attempt = [&]() {
        uint32_t ok;
        if constexpr (CLUSTER)
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(bar), "r"(parity), "r"(1000000u)
                : "memory");
        else
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(bar), "r"(parity), "r"(1000000u)
                : "memory");
        return ok != 0;
    };
    if (attempt()) return true;
    const uint64_t start = globaltimer_ns();
    while (!attempt())
        if (globaltimer_ns() - start > limit_ns) return false;
    return true;
}

// Arrive on a barrier of this CTA.
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One lane of the warp, the same one every time, known to the compiler as one:
// the asynchronous copies and products take their operands from uniform
// registers, and code that several lanes might enter is issued lane by lane.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// ---------------------------------------------------------------------------
// tensor-map copies (TMA).  PAIR: the completion goes to a barrier of either
// CTA of a pair (`bar` is a shared::cluster address).

template <bool PAIR>
__device__ __forceinline__ void tma_2d(uint32_t dst, const void *map, int x, int y, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tma_3d(uint32_t dst, const void *map, int x, int y, int z,
                                       uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

// Four rows of a 2-D tensor chosen by number; a row outside the tensor arrives
// as zeros.
template <bool PAIR>
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void *map, int x, int4 rows,
                                            uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4"
            ".mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::
                "r"(dst),
            "l"(map), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
            "l"(map), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar)
            : "memory");
}

// Address of the same shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    return remote;
}

// Arrive on a barrier of either CTA of a pair, for work that tcgen05 fences order: reads
// of TMEM (waited for, then tcgen05.fence::before_thread_sync) before the products that
// overwrite it (behind fence::after_thread_sync).  So the arrival itself may be relaxed;
// its scope has to hold both CTAs.  A release at cluster scope would also wait for the
// thread's global stores to land (weights' gradient of 128 rows an expert 702 against
// 586 us, in FP32 870 against 740).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t remote_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_bar)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Until at most `N` of this thread's groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------------------
// tensor cores (tcgen05) and their accumulator memory (TMEM)

template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t columns) {
    if constexpr (CTAS == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         dst_smem),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         dst_smem),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <int CTAS>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t columns) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr),
                     "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr),
                     "r"(columns));
}

__device__ __forceinline__ void tcgen05_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tcgen05_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle, `lbo` and `sbo` the byte
// strides of the canonical layout (K-major: sbo between groups of eight rows;
// MN-major: lbo between groups of 64 columns, sbo between groups of eight rows).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return uint64_t{(addr & 0x3FFFFu) >> 4} | (uint64_t{lbo >> 4} << 16) |
           (uint64_t{sbo >> 4} << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// Instruction descriptor: BF16 operands, FP32 accumulators, `a_mn` / `b_mn` for
// an operand stored along M / N.
__device__ __forceinline__ uint32_t instr_desc(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t{a_mn} << 15) | (uint32_t{b_mn} << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool accumulate) {
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(uint32_t{accumulate})
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(uint32_t{accumulate})
            : "memory");
}

// Arrive on `bar` (in both CTAs of a pair) when the issued products are done.
template <int CTAS>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (CTAS == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
}

// 16 accumulator columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 32 accumulator columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

}  // namespace mf
