// Products of few rows per expert with 4-bit weights and group scales.
//
// Bound by the weights' bytes: each is read once for every 32 rows of its
// expert.  A warp takes 32 columns n and up to 32 rows.  It streams 128 summed
// values of its 32 columns a stage (64 bytes a column) through its own ring in
// shared memory (cp.async), turns the nibbles into BF16 integers q - z (exact),
// and multiplies with the rows in mma.m16n8k16, n along M, the rows along N:
// with so few rows the tensor cores only have to keep up with the conversion.
// Each group's FP32 sum is scaled once.  Warps that share a column block split
// the summed values between them and add up through shared memory, in warp order.
#include "experts.cuh"
#include "experts.h"

namespace mf {
namespace {

constexpr int kWarps = 12;
constexpr int kGemvThreads = 32 * kWarps;
constexpr int kCols = 32;      // n of a warp
constexpr int kRowsPass = 32;  // rows of one pass over the weights
constexpr int kSpan = 128;     // summed values of a stage
constexpr int kStages = 4;
// A stage: 32 columns of 64 bytes, 80 apart (the quad reads of eight columns
// then fall into different banks), and per column up to four scales and zeros.
constexpr int kPitch = 80;
constexpr int kScalePitch = 16;  // four FP32 scales, or four BF16 from either half of a word on
constexpr int kZeroPitch = 8;    // four bytes from any byte of a word on
constexpr int kScaleAt = kCols * kPitch;
constexpr int kZeroAt = kScaleAt + kCols * kScalePitch;
constexpr int kStageBytes = kZeroAt + kCols * kZeroPitch;
constexpr int kSumBytes = kCols * kRowsPass * 4;  // one warp's partial results

struct GemvControl {
    int scan[kWarps];
    int tiles[kMaxExperts + 1];
    int lo[kMaxExperts];
    int rows[kMaxExperts];
};

constexpr int kGemvSmem =
    kWarps * (kStages * kStageBytes + kSumBytes) + static_cast<int>(sizeof(GemvControl));
static_assert(kGemvSmem <= 227 * 1024, "shared memory of one CTA");

// 4 bytes global -> shared, the bytes behind `bytes` (0..4) as zeros.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ uint32_t lds_32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    __nv_bfloat162 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = __hsub2(x, y);
    memcpy(&a, &x, 4);
    return a;
}

// Where a warp is in its sequence of (column block, stage) pairs.
struct Cursor {
    int64_t item;
    int stage;    // of the item's spans
    int expert, n0, row0, rows;
    int64_t line;  // expert * n + n0
};

template <int GROUP>
struct Gemv {
    static constexpr int kGroups = kSpan / GROUP;  // of a stage

    const GemvArgs &a;
    const GemvControl &c;
    const int lane, g, t;
    const int share, part;  // warps of a column block, this one's number
    const int64_t first, step, items;
    const int col_blocks, spans, groups;
    const uint32_t ring;
    float *sums;  // of the block's first warp
    const int barrier;

    __device__ void locate(Cursor &p) const {
        if (p.item >= items) return;
        const int u = static_cast<int>(p.item / col_blocks);
        int e = 0;
        for (int s = 512; s > 0; s /= 2)
            if (e + s < a.num_experts && c.tiles[e + s] <= u) e += s;
        p.expert = e;
        p.n0 = static_cast<int>(p.item - int64_t{u} * col_blocks) * kCols;
        const int first_row = (u - c.tiles[e]) * kRowsPass;
        p.row0 = c.lo[e] + first_row;
        p.rows = min(kRowsPass, c.rows[e] - first_row);
        p.line = int64_t{e} * a.n + p.n0;
    }

    __device__ void advance(Cursor &p) const {
        p.stage += share;
        if (p.stage >= spans) {
            p.stage = part;
            p.item += step;
            locate(p);
        }
    }

    // Start the copies of the cursor's stage (nothing behind the last item).
    __device__ void issue(const Cursor &p, uint32_t slot) const {
        if (p.item < items) {
            const int k0 = p.stage * kSpan;
            const uint32_t at = ring + slot * kStageBytes;
            const int half_k = a.k / 2;
            const uint8_t *w = a.w + p.line * half_k + k0 / 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = lane / 4 + 8 * i, chunk = lane % 4;
                const bool in = p.n0 + row < a.n && k0 + chunk * 32 < a.k;
                cp_async_16(at + row * kPitch + chunk * 16,
                            in ? w + int64_t{row} * half_k + chunk * 16 : a.w, in);
            }
            if (p.n0 + lane < a.n) {
                const int g0 = k0 / GROUP;
                const int ng = min(kGroups, groups - g0);
                const int64_t o = (p.line + lane) * groups + g0;
                const uint32_t sd = at + kScaleAt + lane * kScalePitch;
                if (a.scale_fp32) {
                    const float *s = static_cast<const float *>(a.scales) + o;
#pragma unroll
                    for (int i = 0; i < kGroups; ++i)
                        if (i < ng) cp_async_4(sd + 4 * i, s + i, 4);
                } else {
                    // the aligned words that hold the scales
                    const uint8_t *s = static_cast<const uint8_t *>(a.scales) + (o & ~int64_t{1}) * 2;
                    const int bytes = (static_cast<int>(o & 1) + ng) * 2;
#pragma unroll
                    for (int i = 0; i < kGroups / 2 + 1; ++i)
                        if (4 * i < bytes) cp_async_4(sd + 4 * i, s + 4 * i, min(4, bytes - 4 * i));
                }
                if (a.zeros) {
                    const uint8_t *z = a.zeros + (o & ~int64_t{3});
                    const int bytes = static_cast<int>(o & 3) + ng;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (4 * i < bytes)
                            cp_async_4(at + kZeroAt + lane * kZeroPitch + 4 * i, z + 4 * i,
                                       min(4, bytes - 4 * i));
                }
            }
        }
        cp_async_commit();
    }

    __device__ void store(int r, int n, float v) const {
        const int64_t at = r * a.out_ld + n;
        if (a.out_fp32)
            static_cast<float *>(a.out)[at] = v;
        else
            static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
    }

    // One column block with up to 8 NT rows.
    template <int NT>
    __device__ void item(Cursor &now, Cursor &ahead, uint32_t &slot) const {
        const Cursor d = now;
        const __nv_bfloat16 *x[NT];  // the rows this thread feeds (row g of every eight)
        bool live[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int r = 8 * i + g;
            int64_t row = -1;
            if (r < d.rows) row = a.row_index ? __ldg(a.row_index + d.row0 + r) : d.row0 + r;
            live[i] = row >= 0 && row < a.x_rows;
            x[i] = static_cast<const __nv_bfloat16 *>(a.x) + (live[i] ? row * a.x_ld : 0) + 8 * t;
        }
        float acc[2][NT][4] = {};
        while (now.item == d.item) {
            const int k0 = now.stage * kSpan;
            const int blocks = min(kSpan, a.k - k0) / 32;
            uint4 xv[4][NT];
            auto load_x = [&](int b) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    xv[b][i] = live[i] && b < blocks
                                   ? __ldg(reinterpret_cast<const uint4 *>(x[i] + k0 + 32 * b))
                                   : make_uint4(0, 0, 0, 0);
            };
#pragma unroll
            for (int b = 0; b < 4; ++b) load_x(b);
            cp_async_wait<kStages - 2>();
            __syncwarp();
            issue(ahead, (slot + kStages - 1) % kStages);
            advance(ahead);
            const uint32_t at = ring + slot * kStageBytes;
            // element offsets of this stage's first scale, for its place in the copied words
            const int64_t o0 = d.line * groups + k0 / GROUP;
            float sum[2][NT][4];
            uint32_t zero[4] = {0x43084308u, 0x43084308u, 0x43084308u, 0x43084308u};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b >= blocks) break;
                constexpr int kPer = GROUP / 32;
                if (b % kPer == 0) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j) sum[m][i][j] = 0.f;
                    if (a.zeros) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = g + 8 * i;
                            const uint32_t skip =
                                static_cast<uint32_t>(o0 + int64_t{row} * groups) & 3u;
                            const uint32_t z =
                                lds_u8(at + kZeroAt + row * kZeroPitch + skip + b / kPer) & 15u;
                            zero[i] = 0x43004300u | z | (z << 16);
                        }
                    }
                }
                // 0x4300 | q is 128 + q in BF16; minus 128 + z is exact
                uint32_t q[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = lds_32(at + (g + 8 * i) * kPitch + b * 16 + t * 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        q[i][j] = sub_bf16x2(((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u, zero[i]);
                }
                // q[.][j] holds columns j and j + 4 of the thread's eight
                const uint32_t a0[2][4] = {{q[0][0], q[1][0], q[0][1], q[1][1]},
                                           {q[2][0], q[3][0], q[2][1], q[3][1]}};
                const uint32_t a1[2][4] = {{q[0][2], q[1][2], q[0][3], q[1][3]},
                                           {q[2][2], q[3][2], q[2][3], q[3][3]}};
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint4 v = xv[b][i];
                    const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410);
                    const uint32_t b1 = __byte_perm(v.x, v.z, 0x7632);
                    const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410);
                    const uint32_t b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        mma_16816(sum[m][i], a0[m], b0, b1);
                        mma_16816(sum[m][i], a1[m], b2, b3);
                    }
                }
                if (b % kPer == kPer - 1) {
                    float s[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = g + 8 * i;
                        const uint32_t sa = at + kScaleAt + row * kScalePitch;
                        if (a.scale_fp32) {
                            s[i] = __uint_as_float(lds_32(sa + 4 * (b / kPer)));
                        } else {
                            const uint32_t skip =
                                static_cast<uint32_t>(o0 + int64_t{row} * groups) & 1u;
                            s[i] = __uint_as_float(lds_u16(sa + 2 * (skip + b / kPer)) << 16);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                acc[m][i][j] = fmaf(s[2 * m + j / 2], sum[m][i][j], acc[m][i][j]);
                }
            }
            __syncwarp();
            slot = (slot + 1) % kStages;
            advance(now);
        }
        // acc[m][i][j]: n = 16 m + g + 8 (j / 2), row = 8 i + 2 t + j % 2
        if (share == 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int n = 16 * m + g + 8 * (j / 2), r = 8 * i + 2 * t + j % 2;
                        if (r < d.rows && d.n0 + n < a.n) store(d.row0 + r, d.n0 + n, acc[m][i][j]);
                    }
            return;
        }
        float *mine = sums + part * (kCols * kRowsPass);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mine[(8 * i + 2 * t + j % 2) * kCols + 16 * m + g + 8 * (j / 2)] = acc[m][i][j];
        meet();
        if (d.n0 + lane < a.n)
            for (int r = part; r < d.rows; r += share) {
                float v = 0.f;
                for (int s = 0; s < share; ++s) v += sums[s * (kCols * kRowsPass) + r * kCols + lane];
                store(d.row0 + r, d.n0 + lane, v);
            }
        meet();
    }

    // Barrier of the warps that share a column block.
    __device__ void meet() const {
        asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * share) : "memory");
    }
};

template <int GROUP>
__global__ void __launch_bounds__(kGemvThreads, 1)
    grouped_gemv_int4_kernel(const GemvArgs a, const int share) {
    extern __shared__ __align__(16) uint8_t smem[];
    GemvControl &c =
        *reinterpret_cast<GemvControl *>(smem + kWarps * (kStages * kStageBytes + kSumBytes));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_wait();

    // The experts' rows and the numbers of their passes (exclusive scan).
    const int per = (a.num_experts + kGemvThreads - 1) / kGemvThreads;
    const int first = min(static_cast<int>(threadIdx.x) * per, a.num_experts);
    const int last = min(first + per, a.num_experts);
    int sum = 0;
    for (int e = first; e < last; ++e) {
        int lo = 0, hi = static_cast<int>(a.rows);
        if (a.offsets) expert_rows(a.offsets, e, static_cast<int>(a.rows), lo, hi);
        c.lo[e] = lo;
        c.rows[e] = hi - lo;
        c.tiles[e] = sum;
        sum += (hi - lo + kRowsPass - 1) / kRowsPass;
    }
    int before = sum;
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) c.scan[warp] = before;
    before -= sum;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += c.scan[w];
        total += c.scan[w];
    }
    for (int e = first; e < last; ++e) c.tiles[e] += before;
    if (threadIdx.x == 0) c.tiles[a.num_experts] = total;
    __syncthreads();

    const int block = warp / share;
    const int col_blocks = (a.n + kCols - 1) / kCols;
    const Gemv<GROUP> k{a,
                        c,
                        lane,
                        lane / 4,
                        lane % 4,
                        share,
                        warp % share,
                        blockIdx.x + int64_t{gridDim.x} * block,
                        int64_t{gridDim.x} * (kWarps / share),
                        int64_t{total} * col_blocks,
                        col_blocks,
                        (a.k + kSpan - 1) / kSpan,
                        a.k / GROUP,
                        smem_u32(smem) + warp * (kStages * kStageBytes),
                        reinterpret_cast<float *>(smem + kWarps * kStages * kStageBytes) +
                            block * share * (kCols * kRowsPass),
                        1 + block};
    Cursor now{k.first, k.part, 0, 0, 0, 0, 0};
    k.locate(now);
    Cursor ahead = now;
    for (int s = 0; s < kStages - 1; ++s) {
        k.issue(ahead, s);
        k.advance(ahead);
    }
    uint32_t slot = 0;
    while (now.item < k.items) {
        if (now.rows <= 8)
            k.template item<1>(now, ahead, slot);
        else if (now.rows <= 16)
            k.template item<2>(now, ahead, slot);
        else
            k.template item<4>(now, ahead, slot);
    }
    cp_async_wait<0>();
}

template <int GROUP>
cudaError_t launch(const GemvArgs &a, cudaStream_t s) {
    // Warps to a column block: the summed values are split until every warp of the
    // device has work.
    const int64_t blocks = (a.n + kCols - 1) / kCols *
                           (a.rows / kRowsPass + min(int64_t{a.num_experts}, a.rows));
    const int spans = (a.k + kSpan - 1) / kSpan;
    int share = 1;
    while (share < 4 && 2 * share <= spans && blocks * share < int64_t{a.num_sms} * kWarps) share *= 2;
    return launch_ex(grouped_gemv_int4_kernel<GROUP>,
                     dim3(static_cast<unsigned>(min(blocks, int64_t{a.num_sms}))),
                     dim3(kGemvThreads), kGemvSmem, s, 1, a.programmatic, a, share);
}

}  // namespace

cudaError_t prepare_grouped_gemv() {
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(grouped_gemv_int4_kernel<32>, attr, kGemvSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_gemv_int4_kernel<64>, attr, kGemvSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_gemv_int4_kernel<128>, attr, kGemvSmem);
    return e;
}

cudaError_t launch_grouped_gemv_int4(const GemvArgs &a, cudaStream_t s) {
    switch (a.group) {
        case 32: return launch<32>(a, s);
        case 64: return launch<64>(a, s);
        default: return launch<128>(a, s);
    }
}

}  // namespace mf
