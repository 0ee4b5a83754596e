// The 4-bit floating point product grouped by expert on the tensor cores
// (tcgen05, block-scaled):
//
//   D[n, r] = sum over blocks b of sw[n, b] sx[r, b] sum_(k in b) qw[n, k] qx[i(r), k]
//
// computed transposed, as the BF16 products are: a tile's M is 256 output columns over a
// pair of SMs, each holding half of either operand, and its N an expert's rows, any
// multiple of 32 up to 256 (FP32 results 192).  A persistent pair per two SMs walks the
// tiles: a warp copies blocks (TMA, 128-byte swizzle, 256 summed values a step), a warp
// issues the products into one of two accumulators in TMEM, eight warps move the other
// accumulator out, and where rows are gathered, further warps copy them by number.
//
// The scales lie in rows beside the values' rows, and the products read them from TMEM:
// lane l, column c the four bytes of row 32 c + l.  Two teams of four warps read 64 bytes a
// row (a group: four or eight steps; four lanes to a row, the rows 32 apart in one thread),
// write them to shared memory as blocks of 32 lanes by 16 bytes, and the warp that issues
// the products copies a step's blocks into TMEM before it (tcgen05.cp, which runs in order
// with them).
//
// TMEM has 512 columns, and two steps' scales take 96 (E4M3) or 48 of them.  So with 256
// rows the two accumulators overlap: by 96 or 48 columns, which the epilogue moves out
// first, and says so, before the rest.
//
// What bounds it (GB300, 4096 x 4096, short runs): up to some 200 rows an expert the
// weights' bytes (32 experts of 64 rows 51 us, E8M0; 45 at the copy bandwidth).  Beyond, a
// step of 256 rows takes 820 - 830 cycles (E4M3 gathered 940; a launch of 16 experts of 512
// rows, its start and end included), of which the products keep the tensor cores active for
// 512.  Shared memory, at 128 bytes a cycle, is as busy: it brings 32 KB in and reads it once
// more (512 cycles), and writes and reads the scales' blocks (192 cycles, E4M3, or 96).  Which
// waits make up the rest is not measured.  512 rows an expert run at 5.6 (E8M0) and 5.4
// (E4M3) PFLOP/s, gathered 5.2 and 4.8.  Tiles of 192 rows, for which the scales leave whole
// accumulators, ran at 5.2 and 4.3 when 256 did at 5.7 and 4.8.
#include "experts.cuh"
#include "experts.h"
#include "fp4.cuh"
#include "tensor_map.h"

namespace mf {
namespace {

constexpr int kStep = 256;                // summed values per stage: 128 bytes
constexpr int kStepBytes = kStep / 2;
constexpr int kABytes = 128 * kStepBytes;  // A of one CTA and stage
constexpr int kBlockBytes = 512;          // of scales: 32 lanes by 16 bytes, four TMEM columns
constexpr int kTmemColumns = 512;
constexpr int kScanThreads = 256;         // threads that scan the experts
constexpr int kListed = 64;               // tiles of a pair that are found at the start
// Scales of a group, 64 bytes a row: four pieces of 16 bytes a row (one step's, or two), as
// blocks for 128 columns and 256 rows.  The pieces' places are 32 bytes off each other's
// banks: four lanes that have a row's four pieces write them at once.  (Lanes that have four
// rows' same piece need no such gap, but read four times as many lines at once: E4M3, 32768
// rows through 64 experts, 240 against 220 us.)
constexpr int kPieceGap = 32;
constexpr int kPieceBytes = 12 * kBlockBytes + kPieceGap;
constexpr int kGroupBytes = 4 * kPieceBytes;

// FP32 results, and BF16 results of more than kLongSum summed values: the sums leave the
// tensor cores every this many steps and are added up in registers, as the tensor cores
// truncate each partial sum, towards zero: of values of one sign (E4M3 scales) one
// accumulator loses 6.9e-7 of the sum at 4096 values, 4.4e-6 at 16384, 4.3e-5 at 131072 and
// 1.8e-4 at 524288.  Moved every 10 steps it is 2.6e-7 to 3.8e-7 at any of these lengths,
// and 5.8e-8 of 4096 values of either sign.  Up to kLongSum the loss is far below the BF16
// rounding (1.4e-3).
constexpr int kSegment = 10;
constexpr int kLongSum = 131072;

template <int FORMAT>
struct Scales {
    static constexpr int kBytes = FORMAT == kMx ? 8 : 16;     // of a row and step
    static constexpr int kSteps = 64 / kBytes;                // steps of a group
    static constexpr int kWords = kBytes / 4;
    static constexpr int kStepBytes = 3 * kWords * kBlockBytes;  // the columns', the rows'
    static constexpr int kColumns = 12 * kWords;              // of TMEM, of a step
    static constexpr int kColumn = kTmemColumns - 2 * kColumns;  // two steps' in TMEM
};

// What follows from a tile's rows.  SUMS: the sums are moved (kSegment), which takes a
// register for each of a thread's results.
template <bool SUMS>
struct Shape {
    static constexpr int kRows = SUMS ? 192 : 256;  // N of a tile
    static constexpr int kStageBytes = kABytes + kRows / 2 * kStepBytes;
    static constexpr int kStages = SUMS ? 6 : 5;
};

// The second accumulator's first column, and how many it shares with the first.
template <int FORMAT, bool SUMS>
struct Accumulators {
    static constexpr int kSecond = Scales<FORMAT>::kColumn - Shape<SUMS>::kRows;
    static constexpr int kShared = Shape<SUMS>::kRows > kSecond ? Shape<SUMS>::kRows - kSecond : 0;
    static_assert(!SUMS || kShared == 0, "moved sums give whole accumulators back");
};

// Warps: 0 block copies, 1 products, from 4 on eight for the epilogue, then eight for the
// scales, then those that gather (with 2 and 3).
constexpr int kEpilogueWarps = 8;
constexpr int kFirstScale = 4 + kEpilogueWarps;
constexpr int kFirstGather = kFirstScale + 8;

template <bool SUMS, bool GATHER>
struct Warps {
    static constexpr int kGatherWarps = 6;
    static constexpr int kThreads = 32 * (GATHER ? kFirstGather + kGatherWarps - 2 : kFirstGather);
    // With moved sums the epilogue's warps take some of the others' registers
    // (256 * 144 + 384 * 64 = the launch's 640 * 96; 256 * 128 + 512 * 56 = 768 * 80).
    static constexpr int kMany = GATHER ? 128 : 144, kFew = GATHER ? 56 : 64;
    static_assert(kThreads == (GATHER ? 768 : 640) && 256 * kMany + (kThreads - 256) * kFew <=
                                                          kThreads * (GATHER ? 80 : 96),
                  "register split");
};

template <bool SUMS>
struct Control {
    static constexpr int kStages = Shape<SUMS>::kStages;
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], scale_full[2],
        scale_empty[2], shared_empty;
    int4 listed[kListed];        // this pair's first tiles: expert, column, row, rows
    uint32_t tmem;
    int scan[kScanThreads / 32];
    int tiles[kMaxExperts + 1];  // row tiles of the experts before this one
};

template <bool SUMS>
constexpr int kSmemBytes = 1024 + Shape<SUMS>::kStages * Shape<SUMS>::kStageBytes +
                           2 * kGroupBytes + static_cast<int>(sizeof(Control<SUMS>));
static_assert(kSmemBytes<false> <= 227 * 1024 && kSmemBytes<true> <= 227 * 1024,
              "shared memory of one CTA");
static_assert((kMaxExperts + 1) * 4 <= kABytes, "the experts' first rows, at the start");

struct Maps {
    CUtensorMap a, b;  // whole blocks
    CUtensorMap b4;    // rows by number
};

struct Tile {
    int expert;
    int m0;     // first output column
    int row0;   // first output row
    int nrows;  // output rows
    int n;      // nrows rounded up to what the instruction takes
};

__device__ __forceinline__ int round_up(int v, int to) { return (v + to - 1) / to * to; }
__device__ __forceinline__ int divide_up(int v, int by) { return (v + by - 1) / by; }

// A value that all lanes hold alike, known to the compiler as such: what the asynchronous
// instructions take from uniform registers is then computed there, and branches on it do not
// count as divergent.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Tile number t: an expert's column blocks lie behind each other, the row tiles of a block
// together.
template <typename C, typename Lo>
__device__ __forceinline__ int4 locate_tile(const Fp4GemmArgs &a, const C &c, int t,
                                            const Lo &lo) {
    const int mt = divide_up(a.n, 256);
    const int e = expert_of_pass(c.tiles, a.num_experts, 1 << (31 - __clz(a.num_experts)), t / mt);
    const int row0 = lo(e), rows = lo(e + 1) - row0, rt = c.tiles[e + 1] - c.tiles[e];
    const int local = t - c.tiles[e] * mt;
    const int each = round_up(divide_up(rows, rt), 32);  // only the last tile is padded
    const int block = local / rt, first = (local - block * rt) * each;
    return make_int4(e, block * 256, row0 + first, min(each, rows - first));
}

// A pair's tiles in order: every `step`-th one.  The first kListed are found by all threads
// together at the start (a warp that finds one alone takes 0.3 - 0.5 us, once a tile for
// either of the copies and the products: 12 of 75 us at 12 tiles a pair).
template <typename C>
struct Walk {
    const Fp4GemmArgs &a;
    const C &c;
    const int first, step, count;
    int i;

    __device__ Walk(const Fp4GemmArgs &args, const C &control, int tiles)
        : a(args), c(control), first(blockIdx.x / 2), step(gridDim.x / 2),
          count((tiles - first + step - 1) / step), i(0) {}

    __device__ bool more() const { return i < count; }

    // This tile, and on to the next (more() holds).
    __device__ Tile take() {
        int4 t;
        if (i < kListed)
            t = c.listed[i];
        else
            t = locate_tile(a, c, first + i * step, [&](int e) {  // as scan_experts does
                const int rows = static_cast<int>(a.rows);
                if (!a.offsets) return e == 0 ? 0 : rows;
                return min(max(__ldg(a.offsets + e), 0), rows);
            });
        ++i;
        const int rows = uniform(t.w);
        return Tile{uniform(t.x), uniform(t.y), uniform(t.z), rows, round_up(rows, 32)};
    }
};

// Instruction descriptor: E2M1 operands along K, FP32 accumulators, M 256; the first two (or
// four) bytes of a scale's word, with kSecond the other two.
template <int FORMAT>
__device__ __forceinline__ uint32_t fp4_desc(int n) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (uint32_t{FORMAT == kMx} << 23) | (16u << 24);
}
constexpr uint32_t kSecond = (2u << 4) | (2u << 29);

// (a, b: the lower halves of the operands' descriptors, `upper` what they share.)
template <int FORMAT>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a, uint32_t b, uint32_t upper,
                                        uint32_t idesc, uint32_t scale_a, uint32_t scale_b,
                                        bool accumulate) {
    if constexpr (FORMAT == kMx)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %7, 0;\n\t"
            "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %4, [%5], "
            "[%6], p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(upper), "r"(idesc), "r"(scale_a), "r"(scale_b),
            "r"(uint32_t{accumulate})
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %7, 0;\n\t"
            "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %4, "
            "[%5], [%6], p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(upper), "r"(idesc), "r"(scale_a), "r"(scale_b),
            "r"(uint32_t{accumulate})
            : "memory");
}

// Descriptor of a block of scales: groups of eight lanes' 16 bytes lie 128 bytes apart, no
// swizzle.
__device__ __forceinline__ uint64_t block_desc(uint32_t block) {
    return uint64_t{(block & 0x3FFFFu) >> 4} | (uint64_t{128 >> 4} << 16) |
           (uint64_t{128 >> 4} << 32) | (uint64_t{1} << 46);
}

// Such a block to four TMEM columns, the same in each quarter of the lanes, in both CTAs;
// in order with the products.
__device__ __forceinline__ void scales_to_tmem(uint32_t addr, uint32_t block, uint32_t upper) {
    asm volatile(
        "{\n\t.reg .b64 b;\n\tmov.b64 b, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], b;\n\t}" ::"r"(addr),
        "r"(block), "r"(upper)
        : "memory");
}

// A whole warp's wait on a barrier that either CTA of the pair arrives on: all lanes go on,
// or all give up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    uint32_t there;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(there)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__builtin_expect(__all_sync(0xffffffffu, there), 1)) return true;
    return __all_sync(0xffffffffu, mbar_wait_long<true>(bar, parity, limit_ns));
}

// 32 output columns (one per lane) by 16 output rows: a row's 64 or 128 bytes are one store
// of the warp.
template <typename V>
__device__ __forceinline__ void store_rows(const Fp4GemmArgs &a, int64_t out, bool col, int rows,
                                           const V &value) {
    out += threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < 16; ++j, out += a.out_ld)
        if (col && j < rows) {
            if (a.out_fp32)
                static_cast<float *>(a.out)[out] = value(j);
            else
                static_cast<__nv_bfloat16 *>(a.out)[out] = __float2bfloat16_rn(value(j));
        }
}

// The same of 32 rows in BF16, two to a word.
__device__ __forceinline__ void store_pairs(const Fp4GemmArgs &a, int64_t out, bool col, int rows,
                                            const uint32_t (&v)[16]) {
    uint16_t *o = static_cast<uint16_t *>(a.out) + out + threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < 32; ++j, o += a.out_ld)
        if (col && j < rows) *o = static_cast<uint16_t>(v[j / 2] >> (j % 2 * 16));
}

__device__ __forceinline__ void sts_16(uint32_t addr, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

template <int FORMAT, bool GATHER, bool SUMS>
__global__ void __launch_bounds__(Warps<SUMS, GATHER>::kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ Maps maps, const Fp4GemmArgs a) {
    using W = Warps<SUMS, GATHER>;
    using Sc = Scales<FORMAT>;
    using Acc = Accumulators<FORMAT, SUMS>;
    constexpr int kRowsMax = Shape<SUMS>::kRows, kStages = Shape<SUMS>::kStages;
    constexpr int kStageBytes = Shape<SUMS>::kStageBytes;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t groups = base + kStages * kStageBytes;
    auto &c = *reinterpret_cast<Control<SUMS> *>(raw + (groups + 2 * kGroupBytes - smem_u32(raw)));
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const uint32_t full = smem_u32(c.full), empty = smem_u32(c.empty);
    const uint32_t acc_full = smem_u32(c.acc_full), acc_empty = smem_u32(c.acc_empty);
    const uint32_t scale_full = smem_u32(c.scale_full), scale_empty = smem_u32(c.scale_empty);
    const uint32_t shared_empty = smem_u32(&c.shared_empty);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            // the byte count, and all gathering warps: one without a row in a small tile would
            // else fall behind `empty`, whose parity does not tell two phases apart
            mbar_init(full + 8 * i, 1 + (GATHER ? 2 * W::kGatherWarps : 0));
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, kEpilogueWarps * 2);
            mbar_init(scale_full + 8 * i, 4 * 2);
            mbar_init(scale_empty + 8 * i, 1);
        }
        mbar_init(shared_empty, kEpilogueWarps * 2);
        fence_mbar_init();
    }
    // After the wait, not before: a kernel that this one waits for may want TMEM.
    pdl_wait();
    if (warp == 2) tmem_alloc<2>(smem_u32(&c.tmem), kTmemColumns);
    // the experts' first rows lie where the operands will: only the list is made from them
    int *lo = reinterpret_cast<int *>(raw + (base - smem_u32(raw)));
    const int total = scan_experts<kScanThreads>(a.offsets, a.num_experts, static_cast<int>(a.rows),
                                                 kRowsMax, lo, c.tiles, c.scan);
    const int steps = divide_up(a.k, kStep);
    Walk walk(a, c, uniform(divide_up(a.n, 256) * total));
    __syncthreads();
    if (threadIdx.x < min(walk.count, kListed))
        c.listed[threadIdx.x] = locate_tile(a, c, walk.first + threadIdx.x * walk.step,
                                            [&](int e) { return lo[e]; });
    fence_proxy_async_smem();  // before the copies overwrite them
    tcgen05_fence_before();
    __syncthreads();
    cluster_barrier();
    tcgen05_fence_after();
    const uint32_t tmem = uniform(c.tmem);

    bool ok = true;
    if (warp >= 4 && warp < kFirstScale) {
        if constexpr (SUMS)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(W::kMany));
        // Results: lane = output column, TMEM column = output row; eight warps, of which
        // two take the same 32 lanes and every other 32 rows.
        const int w = warp % 4, group = (warp - 4) / 4;
        constexpr int kGroups = kEpilogueWarps / 4;
        const uint32_t done_at = map_to_cta(acc_empty, 0);
        [[maybe_unused]] const uint32_t shared_at = map_to_cta(shared_empty, 0);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
        uint32_t acc_n = 0;  // accumulators taken so far
        while (ok && walk.more()) {
            const Tile d = walk.take();
            const int col0 = d.m0 + rank * 128 + w * 32;
            const bool col = lane < a.n - col0;
            const float factor = a.factor ? __ldg(a.factor + d.expert) : 1.f;
            auto take = [&]() {  // wait for the next accumulator
                ok = warp_wait(acc_full + 8 * (acc_n & 1), acc_n >> 1 & 1, a.timeout_ns);
                tcgen05_fence_after();
                return lanes + (acc_n & 1) * Acc::kSecond;
            };
            auto give_back = [&]() {
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(done_at + 8 * (acc_n & 1));
                ++acc_n;
            };
            if constexpr (SUMS) {
                constexpr int kChunks = kRowsMax / 32 / kGroups;
                float sums[kChunks][32];
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sums[i][j] = 0.f;
                for (int s = 0; s < steps; s += kSegment) {
                    const uint32_t from = take();
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < kChunks; ++i) {
                        const int r = (kGroups * i + group) * 32;
                        if (r < d.nrows) {
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                uint32_t v[16];
                                tmem_ld16(from + r + part * 16, v);
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    sums[i][16 * part + j] += __uint_as_float(v[j]);
                            }
                        }
                    }
                    give_back();
                }
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    const int r = (kGroups * i + group) * 32;
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        if (r + 16 * part < d.nrows)
                            store_rows(a, int64_t{d.row0 + r + 16 * part} * a.out_ld + col0, col,
                                       d.nrows - r - 16 * part,
                                       [&](int j) { return sums[i][16 * part + j] * factor; });
                }
            } else {
                // The columns that the accumulators share are moved first: the first one's
                // last, the second one's first.  32 rows at a time, two of them in BF16 pairs
                // before either is stored, as both may lie there.
                constexpr int kAll = kRowsMax / 32;
                static_assert(Acc::kShared <= 3 * 32, "within the first two of either group's");
                const bool second = acc_n & 1;
                const uint32_t from = take();
                if (!ok) break;
                for (int p = group; p < kAll; p += 2 * kGroups) {
                    uint32_t pairs[2][16];
                    int r[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int at = p + i * kGroups;
                        r[i] = 32 * (second ? at : kAll - 1 - at);
                        if (r[i] >= d.nrows) continue;
                        uint32_t v[32];
                        tmem_ld32(from + r[i], v);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            pairs[i][j] = pack2_rn(__uint_as_float(v[2 * j]) * factor,
                                                   __uint_as_float(v[2 * j + 1]) * factor);
                    }
                    if (p == group) {
                        tcgen05_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(shared_at);
                    }
                    if (p + 2 * kGroups >= kAll) give_back();
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (r[i] < d.nrows)
                            store_pairs(a, int64_t{d.row0 + r[i]} * a.out_ld + col0, col,
                                        d.nrows - r[i], pairs[i]);
                }
            }
        }
    } else {
        if constexpr (SUMS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kFew));
        const uint32_t full_at = map_to_cta(full, 0);
        if (warp == 0) {
            // Copies of whole blocks, and each stage's byte count.
            uint32_t it = 0, stage = 0, phase = 1;
            while (ok && walk.more()) {
                const Tile d = walk.take();
                const int half = d.n / 2;  // B rows of this CTA
                const int b0 = d.row0 + rank * half, m0 = d.m0 + rank * 128;
                const uint32_t bytes = kABytes + round_up(half, GATHER ? 4 : 32) * kStepBytes;
                for (int s = 0; s < steps; ++s, ++it) {
                    // all lanes give up together: the warp meets again below
                    ok = warp_wait(empty + 8 * stage, phase, a.timeout_ns);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t bar = full_at + 8 * stage;
                        const uint32_t sa = base + stage * kStageBytes, sb = sa + kABytes;
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * stage, 2 * bytes);
                        tma_3d<true>(sa, &maps.a, s * kStepBytes, m0, d.expert, bar);
                        if (!GATHER)
#pragma unroll
                            for (int i = 0; i < kRowsMax / 2; i += 32)
                                if (i < half)
                                    tma_2d<true>(sb + i * kStepBytes, &maps.b, s * kStepBytes,
                                                 b0 + i, bar);
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // The products have read every stage (and the other CTA's completions have
            // arrived here) before this CTA may leave.
            if (ok)
                for (uint32_t i = 0; i < kStages && i < it; ++i) {
                    const uint32_t p = it - 1 - i;
                    ok = ok && mbar_wait_long<true>(empty + 8 * (p % kStages), p / kStages & 1,
                                                    a.timeout_ns);
                }
            if (!ok && rank == 0)  // the copies in flight, before the memory is given back
                for (uint32_t i = 0; i < kStages && i < it; ++i) {
                    const uint32_t p = it - 1 - i;
                    (void)mbar_wait_long<true>(full + 8 * (p % kStages), p / kStages & 1,
                                               a.timeout_ns);
                }
        } else if (warp == 1 && rank == 0) {
            // Products.  A step takes the tensor cores 512 cycles, and this warp has to
            // issue its 10 to 16 instructions in less, so the loop is kept short: places are kept
            // by counting, and the last step multiplies its zeros too.
            const uint64_t operands = smem_desc(base, 16, 1024), blocks = block_desc(groups);
            const uint32_t operands_upper = static_cast<uint32_t>(operands >> 32);
            const uint32_t blocks_upper = static_cast<uint32_t>(blocks >> 32);
            constexpr int kRowsFrom = Sc::kWords;  // the rows' first block
            uint32_t stage = 0, phase = 0, acc_n = 0, group_n = 0, scales = tmem + Sc::kColumn;
            const uint32_t turn = scales ^ (scales + Sc::kColumns);
            int before = 0;  // rows of the tile before
            const auto products = [&](const int n) {
                const uint32_t idesc = fp4_desc<FORMAT>(n);
                int in_segment = 0, in_group = 0;
                uint32_t from = 0;
#pragma unroll 1
                for (int left = steps; left > 0; --left) {
                    if (in_group == 0) {
                        if (!warp_wait(scale_full + 8 * (group_n & 1), group_n >> 1 & 1,
                                       a.timeout_ns))
                            return false;
                        from = static_cast<uint32_t>(blocks) + (group_n & 1) * (kGroupBytes / 16);
                    }
                    if (in_segment == 0) {
                        if (!warp_wait(acc_empty + 8 * (acc_n & 1), (acc_n >> 1 & 1) ^ 1,
                                       a.timeout_ns))
                            return false;
                        // The columns shared with the tile before, where either reaches them
                        // (the tile before that has left all its columns, so that the parity
                        // tells).
                        if (Acc::kShared > 0 && (acc_n & 1 ? before : n) > Acc::kSecond &&
                            acc_n > 0 && !warp_wait(shared_empty, (acc_n & 1) ^ 1, a.timeout_ns))
                            return false;
                        before = n;
                    }
                    if (!warp_wait(full + 8 * stage, phase, a.timeout_ns)) return false;
                    tcgen05_fence_after();
                    const uint32_t bar = empty + 8 * stage;
                    const uint32_t da = static_cast<uint32_t>(operands) + stage * (kStageBytes / 16);
                    const uint32_t db = da + kABytes / 16;
                    const uint32_t dst = tmem + (acc_n & 1) * Acc::kSecond;
                    ++in_group;
                    ++in_segment;
                    const bool group_end = left == 1 || in_group == Sc::kSteps;
                    const bool end = left == 1 || (SUMS && in_segment == kSegment);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 3 * Sc::kWords; ++i)
                            scales_to_tmem(scales + 4 * i, from + i * (kBlockBytes / 16),
                                           blocks_upper);
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            // 64 summed values: 32 bytes of a row, a word of its scales or half
                            const int w = FORMAT == kMx ? p / 2 : p;
                            mma_fp4<FORMAT>(dst, da + p * 2, db + p * 2, operands_upper,
                                            FORMAT == kMx && p % 2 ? idesc | kSecond : idesc,
                                            scales + 4 * w, scales + 4 * (kRowsFrom + 2 * w),
                                            p > 0 || in_segment > 1);
                        }
                        mma_commit<2>(bar);
                        if (group_end) mma_commit<2>(scale_empty + 8 * (group_n & 1));
                        if (end) mma_commit<2>(acc_full + 8 * (acc_n & 1));
                    }
                    from += Sc::kStepBytes / 16;
                    if (FORMAT == kNv || in_group % 2 == 0) from += kPieceGap / 16;  // a piece's end
                    scales ^= turn;
                    if (group_end) {
                        in_group = 0;
                        ++group_n;
                    }
                    if (end) {
                        in_segment = 0;
                        ++acc_n;
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                return true;
            };
            while (ok && walk.more()) ok = products(walk.take().n);
            __syncwarp();
        } else if (warp >= kFirstScale && warp < kFirstGather) {
            // Scales.  Two teams of four warps take every other group (a read takes a group's time
            // and more).  A thread takes 16 bytes (a piece) of one row in 32 and of those every
            // 32 behind it: four of the tile's columns, and up to eight of its rows, of which four
            // rows' words make a lane of a block.
            const int team = (warp - kFirstScale) / 4;
            const int row_bytes = a.k / (FORMAT == kMx ? 32 : 16);
            const uint32_t scale_full_at = map_to_cta(scale_full, 0);
            const int groups_of_tile = divide_up(steps, Sc::kSteps);
            const int line = warp % 4 * 8 + lane / 4, piece = lane % 4;
            const uint32_t w_ld = static_cast<uint32_t>(a.ws_ld);  // (below 2^31)
            const uint32_t x_ld = static_cast<uint32_t>(a.xs_ld);
            const int all = walk.count * groups_of_tile;  // (a tile's columns bound both)
            const uint8_t *w_from = nullptr;  // the expert's scales
            int w_row = 0;                    // this thread's first column
            int x_rows[kRowsMax / 32];        // its rows of x, -1: none (zeros)
            uint4 q[12] = {};                 // (blocks are for 256 rows)
            const auto read_16 = [](const uint8_t *base, uint32_t row, uint32_t ld, bool read) {
                const uint8_t *p = base + uint64_t{row} * ld;
                uint4 v;
                asm volatile(
                    "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                    "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
                    "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                    : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
                    : "l"(p), "r"(uint32_t{read}));
                return v;
            };
            auto read_group = [&](int g) {
                const int tile = g / groups_of_tile;
                if (tile >= walk.i) {  // the tile was not taken yet
                    walk.i = tile;
                    const Tile d = walk.take();
                    w_row = d.m0 + static_cast<int>(rank) * 128 + line;
                    w_from = a.w_scales + d.expert * a.ws_expert;
#pragma unroll
                    for (int u = 0; u < kRowsMax / 32; ++u) {
                        const int i = 32 * u + line;
                        int row = -1;
                        if (i < d.nrows) {
                            row = d.row0 + i;
                            if (GATHER) row = __ldg(a.row_index + row);
                            if (row >= a.x_rows) row = -1;
                        }
                        x_rows[u] = row;
                    }
                }
                const int from = (g - tile * groups_of_tile) * 64 + piece * 16;
                const int valid = row_bytes - from;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    q[u] = read_16(w_from + from, w_row + 32 * u, w_ld,
                                   valid > 0 && w_row + 32 * u < a.n);
#pragma unroll
                for (int u = 0; u < kRowsMax / 32; ++u)
                    q[4 + u] = read_16(a.x_scales + from, x_rows[u], x_ld,
                                       valid > 0 && x_rows[u] >= 0);
                if (valid > 0 && valid < 16) {  // what lies behind a row's bytes counts as zeros
                    uint32_t keep[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int bytes = min(max(valid - 4 * j, 0), 4);
                        keep[j] = bytes == 4 ? ~0u : (1u << (8 * bytes)) - 1;
                    }
#pragma unroll
                    for (int u = 0; u < 4 + kRowsMax / 32; ++u) {
                        q[u].x &= keep[0];
                        q[u].y &= keep[1];
                        q[u].z &= keep[2];
                        q[u].w &= keep[3];
                    }
                }
            };
            if (team < all) read_group(team);
            const uint32_t to = groups + team * kGroupBytes + piece * kPieceBytes + line * 16;
            uint32_t n = 0;  // groups of this team so far
            for (int g = team; g < all; g += 2, ++n) {
                ok = warp_wait(scale_empty + 8 * team, (n & 1) ^ 1, a.timeout_ns);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // words of the 16 bytes
                    const int step = j / Sc::kWords, word = j % Sc::kWords;
#pragma unroll
                    for (int b = 0; b < 3; ++b) {
                        const int block = step * 3 * Sc::kWords +
                                          (b == 0 ? word : Sc::kWords + 2 * word + b - 1);
                        const auto w = [&](const uint4 &v) {
                            const uint32_t x = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
                            return FORMAT == kNv ? x & 0x7f7f7f7fu : x;  // without the signs
                        };
                        sts_16(to + block * kBlockBytes, make_uint4(w(q[4 * b]), w(q[4 * b + 1]),
                                                                    w(q[4 * b + 2]), w(q[4 * b + 3])));
                    }
                }
                // The copies to TMEM read this shared memory through the asynchronous proxy,
                // issued by a warp that may be in the other CTA.  So every lane's stores are fenced
                // towards that proxy, gathered by the warp's barrier and released with the
                // arrival, at the pair's scope but for shared memory alone.  A whole release takes
                // some 1 us (512 rows by 32 experts in order, E8M0 and E4M3: 98 and 116 us, gathered
                // 108 and 124; by an idle warp of CTA 1 that passes its teams' arrivals on 98 and
                // 110, 104 and 116; so 97 and 101, 103 and 113).
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_release_smem(scale_full_at + 8 * team);
                if (g + 2 < all) read_group(g + 2);
            }
            // the last group's copies are done, before this CTA may leave
            if (ok && n > 0) ok = warp_wait(scale_empty + 8 * team, (n & 1) ^ 1, a.timeout_ns);
        } else if (GATHER && (warp == 2 || warp == 3 || warp >= kFirstGather)) {
            // Rows by number, four a copy (-1, no such row, arrives as zeros).  Every warp issues
            // some of a step's copies, 80 cycles each: with a warp to a stage, which takes six
            // times as long, the step waits for it.
            constexpr int kQuads = (kRowsMax / 8 + W::kGatherWarps - 1) / W::kGatherWarps;
            const int index = warp < 4 ? warp - 2 : warp - kFirstGather + 2;
            uint32_t stage = 0, phase = 1;
            while (ok && walk.more()) {
                const Tile d = walk.take();
                const int half = d.n / 2, b0 = d.row0 + rank * half;
                const int row_end = d.row0 + d.nrows;
                auto x_row = [&](int i) {
                    const int v = i < row_end ? __ldg(a.row_index + i) : -1;
                    return v >= 0 && v < a.x_rows ? v : -1;
                };
                int4 rows[kQuads];
#pragma unroll
                for (int q = 0; q < kQuads; ++q) {
                    const int i = b0 + 4 * (W::kGatherWarps * q + index);
                    rows[q] = make_int4(x_row(i), x_row(i + 1), x_row(i + 2), x_row(i + 3));
                }
                const int quads = (half / 4 - index + W::kGatherWarps - 1) / W::kGatherWarps;
                for (int s = 0; s < steps; ++s) {
                    ok = warp_wait(empty + 8 * stage, phase, a.timeout_ns);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t bar = full_at + 8 * stage;
                        const uint32_t sb = base + stage * kStageBytes + kABytes + index * 512;
#pragma unroll
                        for (int q = 0; q < kQuads; ++q)
                            if (q < quads)
                                tma_gather4<true>(sb + q * (W::kGatherWarps * 512), &maps.b4,
                                                  s * kStepBytes, rows[q], bar);
                        mbar_arrive_cluster(bar);
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        }
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatusWaitTimeout);
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    cluster_barrier();
    if (warp == 2) {
        tcgen05_fence_after();
        tmem_dealloc<2>(tmem, kTmemColumns);
    }
}

template <int FORMAT, bool GATHER, bool SUMS>
cudaError_t launch(const Maps &maps, const Fp4GemmArgs &a, int64_t tiles, cudaStream_t s) {
    const unsigned ctas = static_cast<unsigned>(2 * min(tiles, int64_t{a.num_pairs}));
    return launch_ex(fp4_gemm_kernel<FORMAT, GATHER, SUMS>, dim3(ctas),
                     dim3(Warps<SUMS, GATHER>::kThreads), kSmemBytes<SUMS>, s, 2, a.programmatic,
                     maps, a);
}

template <int FORMAT, bool GATHER, bool SUMS>
cudaError_t prepare() {
    return cudaFuncSetAttribute(fp4_gemm_kernel<FORMAT, GATHER, SUMS>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<SUMS>);
}

}  // namespace

cudaError_t prepare_fp4_gemm(int *pairs) {
    cudaError_t e = find_encoder();
    if (e == cudaSuccess) e = prepare<kMx, false, false>();
    if (e == cudaSuccess) e = prepare<kMx, false, true>();
    if (e == cudaSuccess) e = prepare<kMx, true, false>();
    if (e == cudaSuccess) e = prepare<kMx, true, true>();
    if (e == cudaSuccess) e = prepare<kNv, false, false>();
    if (e == cudaSuccess) e = prepare<kNv, false, true>();
    if (e == cudaSuccess) e = prepare<kNv, true, false>();
    if (e == cudaSuccess) e = prepare<kNv, true, true>();
    if (e != cudaSuccess) return e;
    // pairs of SMs that run at once: a persistent grid of more would leave some
    // pairs' tiles for a second wave
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(Warps<true, true>::kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<true>;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(pairs, fp4_gemm_kernel<kNv, true, true>, &cfg);
}

cudaError_t launch_fp4_gemm(const Fp4GemmArgs &a, cudaStream_t s) {
    // Few rows of small weights, where latency is all there is (one row through 4096 x 4096:
    // 6.1 us against 8.8 here, through four of 512 x 2048 4.4 against 6.7); twice the weights
    // take as long in either, and eight 4096 x 4096 16 us here, 31 there.
    const int64_t read = min(int64_t{a.num_experts}, a.rows) * a.n * (a.k / 2);
    if (a.rows <= max(8, a.num_experts) && read <= (12 << 20)) return launch_fp4_rows(a, s);
    using u64 = cuuint64_t;
    const u64 bytes = a.k / 2, n = a.n, E = a.num_experts, xr = a.x_rows;
    Maps m = {};
    const auto type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const u64 w_ld = a.w_ld, w_expert = a.w_expert, x_ld = a.x_ld;
    if (!encode_map(&m.a, type, a.w, 3, {bytes, n, E}, {w_ld, w_expert}, kStepBytes, 128) ||
        !encode_map(&m.b, type, a.x, 2, {bytes, xr, 1}, {x_ld, 0}, kStepBytes, 32) ||
        !encode_map(&m.b4, type, a.x, 2, {bytes, xr, 1}, {x_ld, 0}, kStepBytes, 1))
        return cudaErrorInvalidValue;
    // at most this many tiles: the experts' sizes are known on the device only
    const bool sums = a.out_fp32 || a.k > kLongSum, gather = a.row_index != nullptr;
    const int64_t tiles =
        (n + 255) / 256 * (a.rows / (sums ? Shape<true>::kRows : Shape<false>::kRows) +
                           min(int64_t{a.num_experts}, a.rows));
    // tiles are counted in 32 bits (results of so many do not fit into memory)
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    if (a.format == kMx) {
        if (sums)
            return gather ? launch<kMx, true, true>(m, a, tiles, s)
                          : launch<kMx, false, true>(m, a, tiles, s);
        return gather ? launch<kMx, true, false>(m, a, tiles, s)
                      : launch<kMx, false, false>(m, a, tiles, s);
    }
    if (sums)
        return gather ? launch<kNv, true, true>(m, a, tiles, s)
                      : launch<kNv, false, true>(m, a, tiles, s);
    return gather ? launch<kNv, true, false>(m, a, tiles, s)
                  : launch<kNv, false, false>(m, a, tiles, s);
}

}  // namespace mf
