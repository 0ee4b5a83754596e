// moe_grouped_gemm for few rows in all (decode): bound by the weights' bytes, and by
// how evenly they spread over the SMs.
//
// The tensor-core kernel's smallest piece is 128 or 256 columns of an expert, too
// large when a token or two reach a few experts (eight experts of 1024 x 4096: 64 of
// 152 SMs).  Here a warp takes 32 columns and up to 16 rows, streams 64 summed values of
// its columns a stage (128 bytes a column, one tensor-map copy) through its own ring in
// shared memory and multiplies them with the rows in mma.m16n8k16, columns along M;
// where there are few blocks, several warps split one block's summed values and add up
// through shared memory, in warp order.
//
// Measured (GB300, device time): one token through eight 2048 x 4096 matrices 23.4 us
// (5.7 TB/s; 27.0 by the tensor-core kernel), 1024 x 4096 13.7 (21.7), two rows 9 (21); from
// 32 rows on 6.6-7.0 TB/s, the copy's.
#include "experts.h"
#include "few_rows.cuh"
#include "tensor_map.h"

namespace mf {
namespace {

constexpr int kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 32;      // columns of a warp
constexpr int kRowsPass = 16;  // rows of one pass over the weights
constexpr int kSpan = 64;      // summed values of a stage
constexpr int kStages = 4;
constexpr int kStageBytes = kCols * kSpan * 2;

struct RowsControl {
    float sums[kWarps][kRowsPass * kCols];
    uint64_t full[kWarps][kStages];
    int scan[kWarps];
    int passes[kMaxExperts + 1];  // of the experts before this one
    int lo[kMaxExperts + 1];      // first row
};

constexpr int kSmem =
    1024 + kWarps * kStages * kStageBytes + static_cast<int>(sizeof(RowsControl));
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");

struct Rows {
    const GroupedArgs &a;
    const CUtensorMap &map;
    RowsControl &c;
    const int warp, lane, g, t;
    const int share, part;  // warps of a column block, this one's number
    const int block;        // of the CTA
    const int step, items;
    const unsigned col_blocks;
    const int spans, search;
    const uint32_t ring, full;

    __device__ void locate(Cursor &p) const {
        if (p.item >= items) return;
        const int pass = p.item / col_blocks;
        p.expert = expert_of_pass(c.passes, a.num_experts, search, pass);
        p.n0 = (p.item - pass * col_blocks) * kCols;
        p.row0 = c.lo[p.expert] + (pass - c.passes[p.expert]) * kRowsPass;
        p.rows = min(kRowsPass, c.lo[p.expert + 1] - p.row0);
    }

    __device__ void advance(Cursor &p) const {
        p.stage += share;
        if (p.stage >= spans) {
            p.stage = part;
            p.item += step;
            locate(p);
        }
    }

    // Start the copy of a stage (nothing behind the last item) and go on.
    __device__ void issue(Cursor &p, uint32_t slot) const {
        if (p.item >= items) return;
        if (elect_one()) {
            mbar_arrive_expect_tx(full + 8 * slot, kStageBytes);
            tma_3d<false>(ring + slot * kStageBytes, &map, p.stage * kSpan, p.n0, p.expert,
                          full + 8 * slot);
        }
        __syncwarp();
        advance(p);
    }

    __device__ int x_row(const Cursor &d, int r) const {
        const int row = a.row_index ? __ldg(a.row_index + d.row0 + r) : d.row0 + r;
        return row < a.x_rows ? row : -1;
    }

    __device__ void store(const Cursor &d, int r, int n, float v) const {
        const int64_t at = (int64_t{d.row0} + r) * a.out_ld + d.n0 + n;
        if (a.out_fp32)
            static_cast<float *>(a.out)[at] = v;
        else
            static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
    }

    // One column block with up to 8 NT rows.  A copy that does not arrive within `limit`
    // sets the status and the limit to zero: the warp goes on (the others wait for it
    // at the block's barrier), with results of no meaning.
    template <int NT>
    __device__ void item(Cursor &now, Cursor &ahead, uint32_t &it, uint64_t &limit) const {
        const Cursor d = now;
        // The rows this thread feeds (row g of every eight).  Where there is none, any
        // row will do: its results are not stored, or stored as zeros.
        const __nv_bfloat16 *x[NT];
        unsigned outside[NT];  // bit 4 j: row j of every eight is not in x
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int row = x_row(d, min(8 * i + g, d.rows - 1));
            outside[i] = __ballot_sync(0xffffffffu, row < 0);
            x[i] = static_cast<const __nv_bfloat16 *>(a.x) + max(row, 0) * a.x_ld + 8 * t;
        }
        uint4 xv[2][NT];  // the rows' values of the next stage
        auto load_x = [&](int b, int stage) {
            const int k = stage * kSpan + 32 * b;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                xv[b][i] = k + 8 * t < a.k ? __ldg(reinterpret_cast<const uint4 *>(x[i] + k))
                                           : make_uint4(0, 0, 0, 0);
        };
        load_x(0, now.stage);
        load_x(1, now.stage);
        // The tensor cores truncate their partial sums, so every stage's sum is begun anew
        // and added up in FP32 (of 4096 values 1.2e-7 of the result; 5.9e-7 where ten
        // stages made one sum, in the same time).
        float acc[2][NT][4] = {};
        while (now.item == d.item) {
            const uint32_t slot = it % kStages;
            if (limit == 0 ||
                !__all_sync(0xffffffffu, mbar_wait_long(full + 8 * slot, it / kStages & 1, limit))) {
                limit = 0;
                if (lane == 0) atomicOr(a.status, kStatusWaitTimeout);
            }
            issue(ahead, (it + kStages - 1) % kStages);
            const uint32_t w = ring + slot * kStageBytes + g * 128;
            advance(now);
            const int next = now.item == d.item ? now.stage : spans;  // behind the last: zeros
            float sum[2][NT][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // eight summed values of columns g + 8 i (the copy's swizzle keeps the
                // eight columns' words in different banks)
                uint4 q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = lds<uint4>(w + 1024 * i + (((4 * b + t) ^ g) << 4));
                const uint32_t a0[2][4] = {{q[0].x, q[1].x, q[0].y, q[1].y},
                                           {q[2].x, q[3].x, q[2].y, q[3].y}};
                const uint32_t a1[2][4] = {{q[0].z, q[1].z, q[0].w, q[1].w},
                                           {q[2].z, q[3].z, q[2].w, q[3].w}};
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint4 v = xv[b][i];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        if (b == 0)
                            mma_16816_first(sum[m][i], a0[m], v.x, v.y);
                        else
                            mma_16816(sum[m][i], a0[m], v.x, v.y);
                        mma_16816(sum[m][i], a1[m], v.z, v.w);
                    }
                }
                load_x(b, next);
            }
            __syncwarp();
            ++it;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[m][i][j] += sum[m][i][j];
        }
        // acc[m][i][j]: n = 16 m + g + 8 (j / 2), row = 8 i + 2 t + j % 2
        float *mine = c.sums[warp];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = 16 * m + g + 8 * (j / 2);
                    const int r = 8 * i + 2 * t + j % 2;
                    const float v = outside[i] >> (4 * (2 * t + j % 2)) & 1u ? 0.f : acc[m][i][j];
                    if (share > 1)
                        mine[r * kCols + n] = v;
                    else if (r < d.rows && d.n0 + n < a.n)
                        store(d, r, n, v);
                }
        if (share == 1) return;
        meet();
        if (d.n0 + lane < a.n)
            for (int r = part; r < d.rows; r += share) {
                float v = 0.f;
                for (int s = 0; s < share; ++s) v += c.sums[warp - part + s][r * kCols + lane];
                store(d, r, lane, v);
            }
        meet();
    }

    // Barrier of the warps that share a column block.
    __device__ void meet() const {
        asm volatile("bar.sync %0, %1;" ::"r"(block), "r"(32 * share) : "memory");
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    grouped_rows_kernel(const __grid_constant__ CUtensorMap map, const GroupedArgs a,
                        const int share) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + (((smem_u32(raw) + 1023u) & ~1023u) - smem_u32(raw));
    RowsControl &c = *reinterpret_cast<RowsControl *>(smem + kWarps * kStages * kStageBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane < kStages) mbar_init(smem_u32(&c.full[warp][lane]), 1);
    fence_mbar_init();
    pdl_wait();
    const int total = scan_experts<kThreads>(a.offsets, a.num_experts, static_cast<int>(a.rows),
                                             kRowsPass, c.lo, c.passes, c.scan);
    __syncthreads();

    const int block = warp / share;
    const unsigned col_blocks = (a.n + kCols - 1) / kCols;
    const int at_once = kWarps / share, items = total * static_cast<int>(col_blocks);
    const Rows k{a,
                 map,
                 c,
                 warp,
                 lane,
                 lane / 4,
                 lane % 4,
                 share,
                 warp % share,
                 block,
                 static_cast<int>(gridDim.x) * at_once,
                 items,
                 col_blocks,
                 (a.k + kSpan - 1) / kSpan,
                 1 << (31 - __clz(a.num_experts)),
                 smem_u32(smem) + warp * (kStages * kStageBytes),
                 smem_u32(&c.full[warp][0])};
    Cursor now{first_item(block, at_once, items), k.part, 0, 0, 0, 0};
    k.locate(now);
    Cursor ahead = now;
    for (int s = 0; s < kStages - 1; ++s) k.issue(ahead, s);
    uint32_t it = 0;
    uint64_t limit = a.timeout_ns;
    while (now.item < items) {
        if (now.rows <= 8)
            k.template item<1>(now, ahead, it, limit);
        else
            k.template item<2>(now, ahead, it, limit);
    }
    if (limit == 0)  // copies may still be in flight: wait once more before the memory goes
        for (uint32_t s = 1; s <= kStages && s <= it; ++s)
            (void)mbar_wait_long(k.full + 8 * ((it - s) % kStages), (it - s) / kStages & 1,
                                 a.timeout_ns);
}

}  // namespace

cudaError_t prepare_grouped_rows() {
    return cudaFuncSetAttribute(grouped_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmem);
}

cudaError_t launch_grouped_rows(const GroupedArgs &a, cudaStream_t s) {
    using u64 = cuuint64_t;
    CUtensorMap map;
    if (!encode_map(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.w, 3,
                    {static_cast<u64>(a.k), static_cast<u64>(a.n), static_cast<u64>(a.num_experts)},
                    {static_cast<u64>(a.w_ld) * 2, static_cast<u64>(a.w_expert) * 2}, kSpan, kCols))
        return cudaErrorInvalidValue;
    // at most this many column blocks: the experts' sizes are known on the device only
    const int64_t blocks = (a.n + kCols - 1) / kCols *
                           (a.rows / kRowsPass + min(int64_t{a.num_experts}, a.rows));
    const int share = warps_of_block(blocks, (a.k + kSpan - 1) / kSpan, kWarps, a.num_sms);
    return launch_ex(grouped_rows_kernel, dim3(static_cast<unsigned>(min(blocks, int64_t{a.num_sms}))),
                     dim3(kThreads), kSmem, s, 1, a.programmatic, map, a, share);
}

}  // namespace mf
