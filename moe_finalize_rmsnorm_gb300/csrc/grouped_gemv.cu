// Products of few rows per expert with 4-bit weights and group scales.
//
// Bound by the weights' bytes: each is read once for every 16 rows of its
// expert.  A warp takes 32 columns n and up to 16 rows.  It streams 128 summed
// values of its 32 columns a stage (64 bytes a column) through its own ring in
// shared memory (cp.async), turns the nibbles into BF16 integers q - z (exact),
// and multiplies with the rows in mma.m16n8k16, n along M, the rows along N:
// with so few rows the tensor cores only have to keep up with the conversion.
// Each group's FP32 sum is scaled once.  Warps that share a column block split
// the summed values between them and add up through shared memory, in warp order.
#include <string.h>

#include "experts.cuh"
#include "experts.h"

namespace mf {
namespace {

constexpr int kWarps = 12;
constexpr int kGemvThreads = 32 * kWarps;
constexpr int kCols = 32;      // n of a warp
constexpr int kRowsPass = 16;  // rows of one pass over the weights
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

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
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
    int stage;  // of the item's spans
    int expert, n0, row0, rows;
};

// The same for the copies, with this lane's addresses.  Columns behind the last
// one stand for the last one: their results are not stored.
struct Copies {
    int64_t item;
    int stage;
    const uint8_t *w;  // the lane's 16 bytes of the block's first column in this stage
    int at[4];         // and from there to columns lane / 4 + 8 i
    int64_t o;         // number of the first scale of column `lane` in this stage
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
    const uint8_t *ring;
    const uint32_t ring_addr;
    const int search;  // first step of the search for an expert
    float *sums;  // of the block's first warp
    const int barrier;

    // The pass over the weights that holds a column block, counted over the experts.
    __device__ int pass_of(int64_t item) const { return static_cast<int>(item / col_blocks); }

    __device__ int expert_of(int pass) const {
        int e = 0;
        for (int s = search; s > 0; s /= 2)
            if (e + s < a.num_experts && c.tiles[e + s] <= pass) e += s;
        return e;
    }

    __device__ void locate(Cursor &p) const {
        if (p.item >= items) return;
        const int u = pass_of(p.item);
        p.expert = expert_of(u);
        p.n0 = static_cast<int>(p.item - int64_t{u} * col_blocks) * kCols;
        const int first_row = (u - c.tiles[p.expert]) * kRowsPass;
        p.row0 = c.lo[p.expert] + first_row;
        p.rows = min(kRowsPass, c.rows[p.expert] - first_row);
    }

    __device__ void locate(Copies &p) const {
        if (p.item >= items) return;
        const int u = pass_of(p.item);
        const int n0 = static_cast<int>(p.item - int64_t{u} * col_blocks) * kCols;
        const int64_t line = int64_t{expert_of(u)} * a.n + n0;
        p.w = a.w + line * (a.k / 2) + part * (kSpan / 2) + lane % 4 * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) p.at[i] = min(lane / 4 + 8 * i, a.n - 1 - n0) * (a.k / 2);
        p.o = (line + min(lane, a.n - 1 - n0)) * groups + part * kGroups;
    }

    __device__ void advance(Cursor &p) const {
        p.stage += share;
        if (p.stage >= spans) {
            p.stage = part;
            p.item += step;
            locate(p);
        }
    }

    // Start the copies of a stage (nothing behind the last item) and go on.
    __device__ void issue(Copies &p, uint32_t slot) const {
        if (p.item < items) {
            const uint32_t at = ring_addr + slot * kStageBytes;
            const uint32_t wd = at + lane / 4 * kPitch + lane % 4 * 16;
            if (p.stage * kSpan + lane % 4 * 32 < a.k)  // later blocks are not multiplied
#pragma unroll
                for (int i = 0; i < 4; ++i) cp_async_16(wd + 8 * i * kPitch, p.w + p.at[i], true);
            const int ng = min(kGroups, groups - p.stage * kGroups);
            const uint32_t sd = at + kScaleAt + lane * kScalePitch;
            if (a.scale_fp32) {
                const float *s = static_cast<const float *>(a.scales) + p.o;
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
                    if (i < ng) cp_async_4(sd + 4 * i, s + i, 4);
            } else {
                // the aligned words that hold the scales
                const uint8_t *s = static_cast<const uint8_t *>(a.scales) + (p.o & ~int64_t{1}) * 2;
                const int bytes = (static_cast<int>(p.o & 1) + ng) * 2;
#pragma unroll
                for (int i = 0; i < kGroups / 2 + 1; ++i)
                    if (4 * i < bytes) cp_async_4(sd + 4 * i, s + 4 * i, min(4, bytes - 4 * i));
            }
            if (a.zeros) {
                const uint8_t *z = a.zeros + (p.o & ~int64_t{3});
                const int bytes = static_cast<int>(p.o & 3) + ng;
                const uint32_t zd = at + kZeroAt + lane * kZeroPitch;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (4 * i < bytes) cp_async_4(zd + 4 * i, z + 4 * i, min(4, bytes - 4 * i));
            }
            p.stage += share;
            p.w += share * (kSpan / 2);
            p.o += share * kGroups;
            if (p.stage >= spans) {
                p.stage = part;
                p.item += step;
                locate(p);
            }
        }
        cp_async_commit();
    }

    // Row of x that row r of a pass reads, -1 if it is outside.
    __device__ int x_row(const Cursor &d, int r) const {
        const int row = a.row_index ? __ldg(a.row_index + d.row0 + r) : d.row0 + r;
        return row < a.x_rows ? row : -1;
    }

    __device__ void store(const Cursor &d, int r, int n, float v) const {
        if (a.row_index && x_row(d, r) < 0) v = 0.f;  // a row of zeros
        const int64_t at = (int64_t{d.row0} + r) * a.out_ld + d.n0 + n;
        if (a.out_fp32)
            static_cast<float *>(a.out)[at] = v;
        else
            static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
    }

    // One column block with up to 8 NT rows.
    template <int NT>
    __device__ void item(Cursor &now, Copies &ahead, uint32_t &slot) const {
        const Cursor d = now;
        // The rows this thread feeds (row g of every eight).  Where there is none, any
        // row will do: its results are not stored, or stored as zeros.
        const __nv_bfloat16 *x[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int row = x_row(d, min(8 * i + g, d.rows - 1));
            x[i] = static_cast<const __nv_bfloat16 *>(a.x) + max(row, 0) * a.x_ld + 8 * t +
                   now.stage * kSpan;
        }
        // The rows' values of one stage, loaded a stage before they are used: they come
        // from the L2, some 800 cycles away.
        uint4 xv[4][NT];
        auto load_x = [&](int b, int k) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                xv[b][i] = __ldg(reinterpret_cast<const uint4 *>(x[i] + k + 32 * b));
        };
        {
            const int blocks = min(kSpan, a.k - now.stage * kSpan) / 32;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b < blocks) load_x(b, 0);
        }
        // Where the copied words hold the scale and zero of column g + 8 i: from its
        // number modulo 4 on.  (A stage of four groups keeps it, of two moves it by
        // two, of one by one.)
        const unsigned skip0 = static_cast<unsigned>((int64_t{d.expert} * a.n + d.n0 + g) * groups);
        // columns behind the last stand for it
        unsigned skips[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            skips[i] = skip0 + (min(g + 8 * i, a.n - 1 - d.n0) - g) * groups;
        float acc[2][NT][4] = {};
        while (now.item == d.item) {
            const int k0 = now.stage * kSpan;
            const int blocks = min(kSpan, a.k - k0) / 32;
            cp_async_wait<kStages - 2>();
            __syncwarp();
            issue(ahead, (slot + kStages - 1) % kStages);
            const uint8_t *at = ring + slot * kStageBytes;
            const uint8_t *wd = at + g * kPitch + t * 4;
            const unsigned moved = now.stage * kGroups;
            advance(now);
            // blocks of the item's next stage
            const int next = now.item == d.item ? min(kSpan, a.k - now.stage * kSpan) / 32 : 0;
            float sum[2][NT][4];
            uint32_t zero[4] = {0x43084308u, 0x43084308u, 0x43084308u, 0x43084308u};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b >= blocks) break;
                constexpr int kPer = GROUP / 32;  // blocks of a group
                const int group = b / kPer;
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
                            const uint32_t z = at[kZeroAt + (g + 8 * i) * kZeroPitch +
                                                  ((skips[i] + moved) & 3u) + group];
                            zero[i] = __byte_perm(z, 0x43u, 0x4040);  // 128 + z, twice
                        }
                    }
                }
                // 0x4300 | q is 128 + q in BF16; minus 128 + z is exact
                uint32_t q[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w =
                        *reinterpret_cast<const uint32_t *>(wd + 8 * i * kPitch + b * 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        q[i][j] =
                            sub_bf16x2(((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u, zero[i]);
                }
                // q[.][j] holds summed values j and j + 4 of the thread's eight
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
                if (b < next) load_x(b, share * kSpan);
                if (b % kPer == kPer - 1) {
                    float s[4];
                    const uint8_t *sa = at + kScaleAt + g * kScalePitch;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (a.scale_fp32)
                            s[i] = *reinterpret_cast<const float *>(sa + 8 * i * kScalePitch +
                                                                    4 * group);
                        else
                            s[i] = __uint_as_float(
                                uint32_t{*reinterpret_cast<const uint16_t *>(
                                    sa + 8 * i * kScalePitch +
                                    2 * (((skips[i] + moved) & 1u) + group))}
                                << 16);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                acc[m][i][j] =
                                    fmaf(s[2 * m + j / 2], sum[m][i][j], acc[m][i][j]);
                }
            }
            __syncwarp();
            slot = (slot + 1) % kStages;
#pragma unroll
            for (int i = 0; i < NT; ++i) x[i] += share * kSpan;
        }
        // acc[m][i][j]: n = 16 m + g + 8 (j / 2), row = 8 i + 2 t + j % 2
        float *mine = sums + part * (kCols * kRowsPass);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = 16 * m + g + 8 * (j / 2);
                    const int r = 8 * i + 2 * t + j % 2;
                    const float v = acc[m][i][j];
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
                for (int s = 0; s < share; ++s) v += sums[s * (kCols * kRowsPass) + r * kCols + lane];
                store(d, r, lane, v);
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
                        smem + warp * (kStages * kStageBytes),
                        smem_u32(smem) + warp * (kStages * kStageBytes),
                        1 << (31 - __clz(a.num_experts)),
                        reinterpret_cast<float *>(smem + kWarps * kStages * kStageBytes) +
                            block * share * (kCols * kRowsPass),
                        1 + block};
    Cursor now{k.first, k.part, 0, 0, 0, 0};
    k.locate(now);
    Copies ahead{k.first, k.part, nullptr, 0, 0};
    k.locate(ahead);
    for (int s = 0; s < kStages - 1; ++s) k.issue(ahead, s);
    uint32_t slot = 0;
    while (now.item < k.items) {
        if (now.rows <= 8)
            k.template item<1>(now, ahead, slot);
        else
            k.template item<2>(now, ahead, slot);
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
