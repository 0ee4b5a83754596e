// The 4-bit floating point product for few rows of small weights (decode): latency.
//
// A warp takes 32 output columns and up to 8 rows, streams 256 summed values of its
// columns a stage (128 bytes a column, one tensor-map copy) with their scales and the
// rows' through its own ring in shared memory, and multiplies in mma.m16n8k16, columns
// along M, on FP16: E2M1 values are exact there.  A lane takes the eight values of a
// 32-bit word, the four lanes of a quad the 32 of a block:
//
//   E8M0   a block's sum is exact (multiples of 1/4 up to 1152), and so is the product of
//          the two scales within FP32's range: acc += sum * (column's scale * row's scale)
//   E4M3   q * scale is exact in FP16 (6 bits, 2^-10 .. 2688) and is what is multiplied;
//          the tensor cores truncate their partial sums, so every 64 values' sum is begun
//          anew and added up in FP32
//
// Where there are few column blocks, several warps split one block's summed values and
// add up through shared memory, in warp order.
//
// Measured (GB300, device time): one row through 4096 x 4096 6.1 us (E8M0) and 5.4 (E4M3),
// 8.8 by the tensor-core kernel; through four matrices of 512 x 2048 4.4 and 4.0 (6.7).  With
// more weights the instructions count, 25 for a lane's eight weights in ten warps an SM:
// eight of 4096 x 4096 31 us, 16 by the tensor-core kernel.
#include "few_rows.cuh"
#include "fp4.cuh"
#include "tensor_map.h"
#include "experts.h"

namespace mf {
namespace {

constexpr int kCols = 32;   // columns of a warp
constexpr int kSpan = 256;  // summed values of a stage

template <int FORMAT>
struct Fp4Shape {
    static constexpr int kWarps = 10;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = 3;
    static constexpr int kRows = 8;                             // of one pass over the weights
    static constexpr int kScales = FORMAT == kMx ? 8 : 16;      // of a column and stage
    static constexpr int kColBytes = kCols * kSpan / 2;         // a stage's columns
    static constexpr int kWsAt = kRows * kSpan / 2;             // behind the rows: scales
    static constexpr int kXsAt = kWsAt + kCols * kScales;       // and the rows' scales
    static constexpr int kRestBytes = kXsAt + kRows * kScales;  // a stage's rows and scales
    // scales as they are used, of the stage at hand: FP32, or two FP16 to a word
    static constexpr int kTable = 8 * (kCols + kRows);
    struct alignas(16) Control {
        uint8_t rest[kWarps][kStages][kRestBytes];
        uint32_t table[kWarps][kTable];
        float sums[kWarps][kRows * kCols];
        uint64_t full[kWarps][kStages];
        int scan[kWarps];
        int passes[kMaxExperts + 1];  // of the experts before this one
        int lo[kMaxExperts + 1];      // first row
    };
    static constexpr int kSmem =
        1024 + kWarps * kStages * kColBytes + static_cast<int>(sizeof(Control));
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// BYTES (4, 8 or 16) to shared memory, the first `valid` of them from p and zeros behind.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *p, int valid) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(valid)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(p),
                     "n"(BYTES), "r"(valid)
                     : "memory");
}

// Two E4M3 scales (read without their signs) to FP16.
__device__ __forceinline__ uint32_t two_e4m3(uint32_t bytes) {
    uint32_t r;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
        : "=r"(r)
        : "r"(bytes & 0x7f7f));
    return r;
}

template <int FORMAT>
struct Fp4Rows {
    using S = Fp4Shape<FORMAT>;
    const Fp4GemmArgs &a;
    const CUtensorMap &map;
    typename S::Control &c;
    const int warp, lane, g, t;
    const int share, part;  // warps of a column block, this one's number
    const int block;        // of the CTA
    const int step, items;
    const unsigned col_blocks;
    const int spans, search;
    const uint32_t ring, rest, full;

    __device__ void locate(Cursor &p) const {
        if (p.item >= items) return;
        const int pass = p.item / col_blocks;
        p.expert = expert_of_pass(c.passes, a.num_experts, search, pass);
        p.n0 = (p.item - pass * col_blocks) * kCols;
        p.row0 = c.lo[p.expert] + (pass - c.passes[p.expert]) * S::kRows;
        p.rows = min(S::kRows, c.lo[p.expert + 1] - p.row0);
    }

    __device__ void advance(Cursor &p) const {
        p.stage += share;
        if (p.stage >= spans) {
            p.stage = part;
            p.item += step;
            locate(p);
        }
    }

    // The row of x that this lane's row of the pass reads, -1: none (zeros).
    __device__ int x_row(const Cursor &d) const {
        if (d.item >= items || lane >= d.rows) return -1;
        const int row = a.row_index ? __ldg(a.row_index + d.row0 + lane) : d.row0 + lane;
        return row < a.x_rows ? row : -1;
    }

    // Start the copies of a stage (none behind the last item) and go on.  `row`: x_row of
    // the item.
    __device__ void issue(Cursor &p, int &row, uint32_t slot) const {
        if (p.item < items) {
            const uint32_t to = rest + slot * S::kRestBytes;
            if (elect_one()) {
                mbar_arrive_expect_tx(full + 8 * slot, S::kColBytes);
                tma_3d<false>(ring + slot * S::kColBytes, &map, p.stage * (kSpan / 2), p.n0, p.expert, full + 8 * slot);
            }
            __syncwarp();
            const int byte0 = p.stage * (kSpan / 2), left = a.k / 2 - byte0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 4 * i + lane / 8, chunk = lane % 8;
                const int from = __shfl_sync(0xffffffffu, row, r);
                const int valid = from < 0 ? 0 : min(max(left - 16 * chunk, 0), 16);
                cp_async<16>(to + r * 128 + ((chunk ^ (r % 8)) << 4),
                             valid ? a.x + from * a.x_ld + byte0 + 16 * chunk : a.x, valid);
            }
            constexpr int kBlock = FORMAT == kMx ? 32 : 16;
            const int s0 = p.stage * S::kScales, s_left = min(a.k / kBlock - s0, S::kScales);
            const int n = p.n0 + lane;
            const bool col = n < a.n;
            cp_async<S::kScales>(to + S::kWsAt + lane * S::kScales,
                                 col ? a.w_scales + p.expert * a.ws_expert + n * a.ws_ld + s0
                                     : a.w_scales,
                                 col ? s_left : 0);
            if (lane < S::kRows)
                cp_async<S::kScales>(to + S::kXsAt + lane * S::kScales,
                                     row >= 0 ? a.x_scales + row * a.xs_ld + s0 : a.x_scales,
                                     row >= 0 ? s_left : 0);
            const int item = p.item;
            advance(p);
            if (p.item != item) row = x_row(p);
        }
        cp_async_commit();
    }

    __device__ void store(const Cursor &d, int r, int n, float v) const {
        if (a.factor) v *= __ldg(a.factor + d.expert);
        const int64_t at = (int64_t{d.row0} + r) * a.out_ld + d.n0 + n;
        if (a.out_fp32)
            static_cast<float *>(a.out)[at] = v;
        else
            static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
    }

    // The stage's scales as they are used: word b of line i (a column, then the rows).
    // MX: the block's scale in FP32; NV: the two blocks' of 32 values in FP16.
    __device__ void convert_scales(uint32_t from) const {
        uint32_t *to = c.table[warp];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i == 1 && lane >= S::kRows) break;
            const uint32_t at = from + (i ? S::kXsAt : S::kWsAt) + lane * S::kScales;
            uint32_t words[S::kScales / 4], v[8];
            if constexpr (FORMAT == kMx) {
                const uint2 q = lds<uint2>(at);
                words[0] = q.x;
                words[1] = q.y;
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    v[b] = __float_as_uint(scale_of<kMx>(words[b / 4] >> (8 * (b % 4)) & 255u));
            } else {
                const uint4 q = lds<uint4>(at);
                words[0] = q.x;
                words[1] = q.y;
                words[S::kScales / 4 - 2] = q.z;
                words[S::kScales / 4 - 1] = q.w;
#pragma unroll
                for (int b = 0; b < 8; ++b) v[b] = two_e4m3(words[b / 2] >> (16 * (b % 2)));
            }
            // 16-byte pieces, a line's two in turned places: lines 0..7's first pieces lie in
            // different banks
            const int line = 32 * i + lane;
            uint4 *o = reinterpret_cast<uint4 *>(to + 8 * line);
            o[(line >> 2) & 1] = make_uint4(v[0], v[1], v[2], v[3]);
            o[((line >> 2) & 1) ^ 1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
        __syncwarp();
    }

    // Four words (b = 4 half ..) of a line.
    __device__ uint4 scales(int line, int half) const {
        return *reinterpret_cast<const uint4 *>(c.table[warp] + 8 * line +
                                                4 * (((line >> 2) & 1) ^ half));
    }

    // One column block with up to 8 rows.  A copy that does not arrive within `limit`
    // sets the status and the limit to zero: the warp goes on (the others wait for it at
    // the block's barrier), with results of no meaning.
    __device__ void item(Cursor &now, Cursor &ahead, int &row, uint32_t &it,
                         uint64_t &limit) const {
        const Cursor d = now;
        float acc[2][4] = {};
        while (now.item == d.item) {
            const uint32_t slot = it % S::kStages;
            cp_async_wait<S::kStages - 2>();
            if (limit == 0 ||
                !__all_sync(0xffffffffu, mbar_wait_long(full + 8 * slot, it / S::kStages & 1, limit))) {
                limit = 0;
                if (lane == 0) atomicOr(a.status, kStatusWaitTimeout);
            }
            __syncwarp();  // every lane's copies are there, and the stage before is read
            issue(ahead, row, (it + S::kStages - 1) % S::kStages);
            const uint32_t w = ring + slot * S::kColBytes, x = rest + slot * S::kRestBytes;
            convert_scales(x);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // MX: columns g + 8 i, and the rows 2 t and 2 t + 1 of the results; NV: the
                // columns and the row g that this lane feeds
                uint4 sw[4], sx[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) sw[i] = scales(g + 8 * i, half);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    sx[j] = scales(kCols + (FORMAT == kMx ? 2 * t + j : g), half);
                const auto word = [](const uint4 &v, int i) {
                    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
                };
                float sum[2][4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t at = g * 128 + (((4 * half + b) ^ g) << 4) + 4 * t;
                    uint32_t wv[4][4], xv[4];
                    const uint32_t pick = t < 2 ? 0x1010u : 0x3232u;  // NV: this lane's block
#pragma unroll
                    for (int i = 0; i < 5; ++i) {
                        uint32_t(&v)[4] = i < 4 ? wv[i < 4 ? i : 0] : xv;
                        from_e2m1(lds<uint32_t>(at + (i < 4 ? w + 1024 * i : x)), v);
                        if (FORMAT == kNv) {
                            const uint32_t s = __byte_perm(
                                word(i < 4 ? sw[i < 4 ? i : 0] : sx[0], b), 0, pick);
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[j] = hmul2(v[j], s);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint32_t a0[4] = {wv[2 * m][0], wv[2 * m + 1][0], wv[2 * m][1],
                                                wv[2 * m + 1][1]};
                        const uint32_t a1[4] = {wv[2 * m][2], wv[2 * m + 1][2], wv[2 * m][3],
                                                wv[2 * m + 1][3]};
                        if (FORMAT == kMx || b % 2 == 0)
                            mma_f16_first(sum[m], a0, xv[0], xv[1]);
                        else
                            mma_f16(sum[m], a0, xv[0], xv[1]);
                        mma_f16(sum[m], a1, xv[2], xv[3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (FORMAT == kMx)
                                acc[m][j] =
                                    fmaf(sum[m][j],
                                         __uint_as_float(word(sw[2 * m + j / 2], b)) *
                                             __uint_as_float(word(sx[j % 2], b)),
                                         acc[m][j]);
                            else if (b % 2 == 1)
                                acc[m][j] += sum[m][j];
                        }
                    }
                }
            }
            advance(now);
            __syncwarp();
            ++it;
        }
        // acc[m][j]: n = 16 m + g + 8 (j / 2), row = 2 t + j % 2
        float *mine = c.sums[warp];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = 16 * m + g + 8 * (j / 2), r = 2 * t + j % 2;
                if (share > 1)
                    mine[r * kCols + n] = acc[m][j];
                else if (r < d.rows && d.n0 + n < a.n)
                    store(d, r, n, acc[m][j]);
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

template <int FORMAT>
__global__ void __launch_bounds__(Fp4Shape<FORMAT>::kThreads, 1)
    fp4_rows_kernel(const __grid_constant__ CUtensorMap map, const Fp4GemmArgs a, const int share) {
    using S = Fp4Shape<FORMAT>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + (((smem_u32(raw) + 1023u) & ~1023u) - smem_u32(raw));
    auto &c = *reinterpret_cast<typename S::Control *>(smem + S::kWarps * S::kStages * S::kColBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane < S::kStages) mbar_init(smem_u32(&c.full[warp][lane]), 1);
    fence_mbar_init();
    pdl_wait();
    const int total = scan_experts<S::kThreads>(a.offsets, a.num_experts, static_cast<int>(a.rows),
                                                S::kRows, c.lo, c.passes, c.scan);
    __syncthreads();

    const int block = warp / share;
    const unsigned col_blocks = (a.n + kCols - 1) / kCols;
    const int at_once = S::kWarps / share, items = total * static_cast<int>(col_blocks);
    const Fp4Rows<FORMAT> k{a,
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
                                smem_u32(smem) + warp * (S::kStages * S::kColBytes),
                                smem_u32(c.rest[warp]),
                                smem_u32(&c.full[warp][0])};
    Cursor now{first_item(block, at_once, items), k.part, 0, 0, 0, 0};
    k.locate(now);
    Cursor ahead = now;
    int row = k.x_row(ahead);
    for (int s = 0; s < S::kStages - 1; ++s) k.issue(ahead, row, s);
    uint32_t it = 0;
    uint64_t limit = a.timeout_ns;
    while (now.item < items) k.item(now, ahead, row, it, limit);
    cp_async_wait<0>();
    if (limit == 0)  // copies may still be in flight: wait once more before the memory goes
        for (uint32_t s = 1; s <= S::kStages && s <= it; ++s)
            (void)mbar_wait_long(k.full + 8 * ((it - s) % S::kStages), (it - s) / S::kStages & 1,
                                 a.timeout_ns);
}

template <int FORMAT>
cudaError_t launch(const Fp4GemmArgs &a, cudaStream_t s) {
    using S = Fp4Shape<FORMAT>;
    using u64 = cuuint64_t;
    CUtensorMap map;
    if (!encode_map(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, 3,
                    {static_cast<u64>(a.k / 2), static_cast<u64>(a.n),
                     static_cast<u64>(a.num_experts)},
                    {static_cast<u64>(a.w_ld), static_cast<u64>(a.w_expert)}, kSpan / 2, kCols))
        return cudaErrorInvalidValue;
    // at most this many column blocks: the experts' sizes are known on the device only
    const int64_t blocks = (a.n + kCols - 1) / kCols *
                           (a.rows / S::kRows + min(int64_t{a.num_experts}, a.rows));
    if (blocks > INT32_MAX / 2) return cudaErrorInvalidValue;  // they are counted in 32 bits
    const int share = warps_of_block(blocks, (a.k + kSpan - 1) / kSpan, S::kWarps, a.num_sms);
    return launch_ex(fp4_rows_kernel<FORMAT>,
                     dim3(static_cast<unsigned>(min(blocks, int64_t{a.num_sms}))),
                     dim3(S::kThreads), S::kSmem, s, 1, a.programmatic, map, a, share);
}

template <int FORMAT>
cudaError_t prepare() {
    return cudaFuncSetAttribute(fp4_rows_kernel<FORMAT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Fp4Shape<FORMAT>::kSmem);
}

}  // namespace

cudaError_t prepare_fp4_rows() {
    cudaError_t e = find_encoder();
    if (e == cudaSuccess) e = prepare<kMx>();
    if (e == cudaSuccess) e = prepare<kNv>();
    return e;
}

cudaError_t launch_fp4_rows(const Fp4GemmArgs &a, cudaStream_t s) {
    return a.format == kMx ? launch<kMx>(a, s) : launch<kNv>(a, s);
}

}  // namespace mf
