// Matrix products grouped by expert: forward, and the gradients of the rows
// and of the weights, on the tensor cores.
//
// Every product is computed transposed: a tile's M is the output's columns and
// its N the output's rows,
//
//   forward  D[n, r] = sum_k W[e][n, k] x[i(r), k]
//   dgrad    D[k, r] = sum_n W[e][n, k] dy[r, n]
//   wgrad    D[k, n] = sum_r x[i(r), k] dy[r, n]
//
// so the ragged dimension of the first two, an expert's rows, is the one whose
// tile may be any multiple of 32 up to 256 (16 for a single CTA): an expert of 40
// rows costs 64, not 128 or 256.  An expert's rows are split into tiles of one such
// multiple, the last with what is left (528 rows: 192, 192 and 144).  In wgrad the
// ragged dimension is the summed one; the step that holds an expert's last rows
// reads them by number, and the rows behind them as zeros, so that a row of
// another expert (or one that was never written) enters nothing.
//
// One persistent CTA (or pair of CTAs: one tile of 256 columns over two SMs,
// each holding half of either operand) per SM walks the tiles: a warp that
// issues the copies of blocks (TMA, 128-byte swizzle, 64 summed values a step), a
// warp that issues the products into one of two accumulators in TMEM, four or
// eight warps that move the other accumulator out, and six or twelve for rows that
// are gathered.
//
// What bounds it (4096 x 4096, up to 16384 rows, GB300, short runs): up to some 200
// rows an expert the weights' bytes (64 experts: 330-354 us, 317 at the copy
// bandwidth).  Beyond, a step of a tile of N rows brings (16 KB + 64 N) into an SM, which
// takes in 64 bytes a cycle, for 2 N cycles of products: the two are equal at N = 256
// and the copies take longer below.  So 512 and 1024 rows (tiles of 256) run at 1.7-1.87
// PFLOP/s, as a plain library product, 288 (160 and 128) at 1.25 and 528 (192, 192 and
// 144) at 1.45-1.53, where the bytes allow 1.35 and 1.52.  The weights' gradient has
// tiles of 256 always and is bound by its results' way out where few rows are summed:
// 128 rows 0.47, 288 0.9, 512 1.24, 528 1.1-1.17, 1024 1.7-1.78 PFLOP/s.
// Tiles of two blocks that share an operand needed fewer and
// longer stages and both accumulators: 6 % faster at 288 rows, 4-30 % slower from
// 512 rows on and for the weights' gradient; not kept.
#include "experts.cuh"
#include "experts.h"
#include "tensor_map.h"

namespace mf {
namespace {

constexpr int kRowsMax = 256;               // N of a tile
constexpr int kStep = 64;                   // summed values per stage: 128 bytes of BF16
constexpr int kABytes = 128 * kStep * 2;    // A of one CTA and stage
constexpr int kStagesBytes = 192 * 1024;
constexpr int kTmemColumns = 512;           // two accumulators of 256
constexpr int kTurnBytes = 2048;            // an epilogue warp's block to turn results in
constexpr int kScanThreads = 256;           // threads that scan the experts

// Moved sums: moved out of TMEM and added up in registers every this many steps.  The
// tensor cores truncate each partial sum, an error that grows with the products added to
// one accumulator: every 16 summed values lose up to 9e-8 of it, towards zero (values of
// one sign: 4096 of them 1.1e-5 of the sum, 32768 1.6e-4, 2^20 6.1e-3; of either sign the
// losses cancel for the most part).  640 summed values keep it near 1e-6 for values of
// one sign; of either sign FP32 results are off by 5.8e-7 of the result (320 values
// 2.9e-7, as FP32 multiply-adds, in 1-3 % more time, the weights' gradient 5-8 %).
constexpr int kSegment = 10;
// BF16 results of more than this many summed values are, too.  Up to it one accumulator
// takes the whole sum: 1.6e-4 beside the rounding's 2^-8.
constexpr int kLongSum = 32768;

template <int CTAS>
struct Shape {
    static constexpr int kM = 128 * CTAS;
    static constexpr int kStageBytes = kABytes + kRowsMax / CTAS * kStep * 2;
    static constexpr int kStages = kStagesBytes / kStageBytes;  // 6, a single CTA 4
};

// Warps: 0 block copies, 1 products, from 4 on the epilogue, then those that gather
// (with 2 and 3, which otherwise only copy the last rows of a sum).
// SUMS: the sums are moved (kSegment).
template <int CTAS, bool SUMS, bool GATHER>
struct Warps {
    static constexpr int kEpilogue = SUMS ? 8 : 4;
    static constexpr int kFirstGather = 4 + kEpilogue;
    static constexpr int kShare = SUMS ? 1 : 2;  // gathering warps of a stage
    // 512 threads with moved sums: whole warpgroups, as the register split needs
    static constexpr int kAll = !GATHER ? kFirstGather
                                : SUMS  ? 16
                                        : kFirstGather + kShare * Shape<CTAS>::kStages - 2;
    static constexpr int kThreads = 32 * kAll;
};

// Shared memory behind the stages and the epilogue's blocks.
struct Control {
    int4 list[256];              // rows by number, four a copy; a part for each gathering warp
    uint64_t full[6], empty[6], tail[6], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int scan[kScanThreads / 32];
    int tiles[kMaxExperts + 1];  // row tiles of the experts before this one; wgrad: rows summed
    int lo[kMaxExperts + 1];     // first row; the next expert's is the end
};

constexpr int kSmemBytes = 1024 + kStagesBytes + 8 * kTurnBytes + sizeof(Control);
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");

struct Maps {
    CUtensorMap a, b;    // whole blocks
    CUtensorMap a4, b4;  // rows by number
};

struct Tile {
    int expert;
    int m0;       // first output column
    int row0;     // first output row (forward, dgrad: of the buffer; wgrad: n)
    int nrows;    // output rows
    int n;        // nrows rounded up to what the instruction takes
    int steps;    // of 64 summed values
    int summed;   // summed values
    int sum0;     // wgrad: first row of the expert
};

__device__ __forceinline__ int round_up(int v, int to) { return (v + to - 1) / to * to; }
__device__ __forceinline__ int divide_up(int v, int by) { return (v + by - 1) / by; }

template <int KIND, int CTAS>
__device__ __forceinline__ Tile tile_of(const GroupedArgs &a, const Control &c, int t) {
    constexpr int M = Shape<CTAS>::kM;
    const int mt = divide_up(KIND == kForward ? a.n : a.k, M);
    Tile r;
    if (KIND == kWgrad) {
        const int nt = divide_up(a.n, kRowsMax);
        r.expert = t / (mt * nt);
        const int local = t - r.expert * (mt * nt);
        r.m0 = local % mt * M;
        r.row0 = local / mt * kRowsMax;
        r.nrows = min(kRowsMax, a.n - r.row0);
        r.summed = c.tiles[r.expert];
        r.sum0 = c.lo[r.expert];
    } else {
        const int u = t / mt;
        const int e = expert_of_pass(c.tiles, a.num_experts, kMaxExperts / 2, u);
        r.expert = e;
        const int rows = c.lo[e + 1] - c.lo[e];
        const int rt = c.tiles[e + 1] - c.tiles[e];
        const int local = t - c.tiles[e] * mt;
        // of what the instruction takes: only the last tile is padded
        const int each = round_up(divide_up(rows, rt), 16 * CTAS);
        const int first = local % rt * each;
        r.m0 = local / rt * M;
        r.row0 = c.lo[e] + first;
        r.nrows = min(each, rows - first);
        r.summed = KIND == kForward ? a.k : a.n;
        r.sum0 = 0;
    }
    r.n = round_up(r.nrows, 16 * CTAS);
    r.steps = divide_up(r.summed, kStep);
    return r;
}

// 32 output columns (one per lane) by 16 output rows in FP32 to rows of `out`:
// turned in the warp's block of shared memory, 128 bytes a row (or 64 of BF16).
// `out` is the first row's first column, `cols` and `rows` what exists of the block.
template <typename V>
__device__ __forceinline__ void store16(const GroupedArgs &a, uint8_t *block, int64_t out, int64_t ld,
                                        int cols, int rows, const V &value) {
    const int lane = threadIdx.x % 32;
    float *f = reinterpret_cast<float *>(block);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j * 32 + lane] = value(j);
    __syncwarp();
    if (a.out_fp32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 4 + lane / 8, col = lane % 8 * 4;
            if (r >= rows || col >= cols) continue;
            float4 x = *reinterpret_cast<float4 *>(f + r * 32 + col);
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + out + r * ld + col);
            if (a.accumulate) {
                const float4 y = *o;
                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            *o = x;
        }
    } else {  // BF16 of a long sum, or that is added to: rounded once
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 8 + lane / 4, col = lane % 4 * 8;
            if (r >= rows || col >= cols) continue;
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + out + r * ld +
                                                 col);
            float y[8];
            unpack8(a.accumulate ? *o : make_uint4(0, 0, 0, 0), y);
#pragma unroll
            for (int u = 0; u < 8; ++u) y[u] += f[r * 32 + col + u];
            *o = pack8_rn(y);
        }
    }
}

// The same of 32 rows in BF16.
__device__ __forceinline__ void store32_bf16(const GroupedArgs &a, uint8_t *block, int64_t out,
                                             int64_t ld, int cols, int rows,
                                             const uint32_t (&v)[32]) {
    const int lane = threadIdx.x % 32;
    __nv_bfloat16 *h = reinterpret_cast<__nv_bfloat16 *>(block);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j) h[j * 32 + lane] = __float2bfloat16_rn(__uint_as_float(v[j]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 4, col = lane % 4 * 8;
        if (r < rows && col < cols)
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + out + r * ld + col) =
                *reinterpret_cast<uint4 *>(h + r * 32 + col);
    }
}

// Rows i to i + 3, -1 (zeros) from `end` on.
__device__ __forceinline__ int4 rows_until(int i, int end) {
    return make_int4(i < end ? i : -1, i + 1 < end ? i + 1 : -1, i + 2 < end ? i + 2 : -1,
                     i + 3 < end ? i + 3 : -1);
}

// wgrad: the columns [b0, b0 + half) of a step's last rows of dy, every `share`-th
// four rows from the `sub`-th on.
template <bool PAIR>
__device__ __forceinline__ void dy_tail(const Maps &maps, uint32_t sb, int r0, int end, int b0,
                                        int half, int sub, int share, uint32_t bar) {
    for (int q = sub; q < kStep / 4; q += share)
        for (int at = 0; at < half; at += 64)
            tma_gather4<PAIR>(sb + at / 64 * 8192 + q * 512, &maps.b4, b0 + at,
                              rows_until(r0 + 4 * q, end), bar);
}

template <int KIND, int CTAS, bool GATHER, bool SUMS>
__global__ void __launch_bounds__(Warps<CTAS, SUMS, GATHER>::kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ Maps maps, const GroupedArgs a) {
    using S = Shape<CTAS>;
    using W = Warps<CTAS, SUMS, GATHER>;
    constexpr bool PAIR = CTAS == 2;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t *blocks = raw + (base - smem_u32(raw)) + kStagesBytes;
    Control &c = *reinterpret_cast<Control *>(blocks + 8 * kTurnBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const uint32_t full = smem_u32(c.full), empty = smem_u32(c.empty), tail = smem_u32(c.tail);
    const uint32_t acc_full = smem_u32(c.acc_full), acc_empty = smem_u32(c.acc_empty);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
            mbar_init(tail + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, W::kEpilogue * CTAS);
        }
        fence_mbar_init();
    }
    // After the wait, not before: a kernel that this one waits for may want TMEM.
    pdl_wait();
    if (warp == 2) tmem_alloc<CTAS>(smem_u32(&c.tmem), kTmemColumns);

    const int total = scan_experts<kScanThreads>(a.offsets, a.num_experts, static_cast<int>(a.rows),
                                                 kRowsMax, c.lo, c.tiles, c.scan);
    if (KIND == kWgrad) {  // by the thread that scanned the expert
        const int per = divide_up(a.num_experts, kScanThreads);
        const int first = min(static_cast<int>(threadIdx.x) * per, a.num_experts);
        for (int e = first; e < min(first + per, a.num_experts); ++e) {
            const int rows = max(c.lo[e + 1] - c.lo[e], 0);
            c.tiles[e] = rows >= a.sum_from && rows <= a.sum_to ? rows : 0;
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    if (PAIR) cluster_barrier();
    tcgen05_fence_after();
    const uint32_t tmem = c.tmem;

    const int columns = KIND == kForward ? a.n : a.k;
    const int mt = divide_up(columns, S::kM);
    int tiles = mt * (KIND == kWgrad ? a.num_experts * divide_up(a.n, kRowsMax) : total);
    if (KIND == kWgrad && SUMS && a.sum_from > 0) {  // seldom has any expert so many rows
        bool any = false;
        for (int e = threadIdx.x; e < a.num_experts; e += W::kThreads)
            any |= c.tiles[e] > 0;
        if (!__syncthreads_or(any)) tiles = 0;
    }
    const int first_tile = blockIdx.x / CTAS, tile_step = gridDim.x / CTAS;

    // Registers: the warps that hold the moved sums take some of the others'
    // (8 * 32 * 176 + 8 * 32 * 80 = the launch's 512 * 128).
    constexpr bool kMoveRegisters = SUMS && GATHER;
    static_assert(!kMoveRegisters || W::kThreads == 512, "register split");

    if (warp >= 4 && warp < W::kFirstGather) {
        if constexpr (kMoveRegisters) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        // Results: lane = output column, TMEM column = output row; four warps (one
        // per 32 lanes) to all TMEM columns, or eight to every other 32.
        const int w = warp % 4, group = (warp - 4) / 4;
        constexpr int kGroups = W::kEpilogue / 4;
        uint8_t *block = blocks + (warp - 4) * kTurnBytes;
        const uint32_t done_at = PAIR ? map_to_cta(acc_empty, 0) : acc_empty;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
        uint32_t acc_n = 0;  // accumulators taken so far
        bool ok = true;
        for (int t = first_tile; t < tiles && ok; t += tile_step) {
            const Tile d = tile_of<KIND, CTAS>(a, c, t);
            const bool none = d.steps == 0;
            // nothing to add, or another launch's
            if (none && (a.accumulate || c.lo[d.expert + 1] > c.lo[d.expert])) continue;
            const int64_t ld = KIND == kWgrad ? a.k : a.out_ld;
            const int64_t row0 = KIND == kWgrad ? int64_t{d.expert} * a.n + d.row0 : d.row0;
            const int col0 = d.m0 + rank * 128 + w * 32;
            const int cols = columns - col0;  // what exists of the warp's 32
            auto take = [&]() {  // wait for the next accumulator
                ok = __all_sync(0xffffffffu, mbar_wait_long<PAIR>(acc_full + 8 * (acc_n & 1),
                                                            acc_n >> 1 & 1, a.timeout_ns));
                tcgen05_fence_after();
                return lanes + (acc_n & 1) * kRowsMax;
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
                for (int s = 0; s < d.steps; s += kSegment) {
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
                            store16(a, block, (row0 + r + 16 * part) * ld + col0, ld, cols,
                                    d.nrows - r - 16 * part,
                                    [&](int j) { return sums[i][16 * part + j]; });
                }
            } else {
                const uint32_t from = none ? 0 : take();
                if (!ok) break;
                for (int r = group * 32; r < d.nrows; r += kGroups * 32) {
                    uint32_t v[32];
                    if (none) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0;
                    } else {
                        tmem_ld32(from + r, v);
                    }
                    const int64_t out = (row0 + r) * ld + col0;
                    if (!(KIND == kWgrad && a.accumulate)) {
                        store32_bf16(a, block, out, ld, cols, d.nrows - r, v);
                    } else {
#pragma unroll
                        for (int part = 0; part < 2; ++part)
                            if (r + 16 * part < d.nrows)
                                store16(a, block, out + 16 * part * ld, ld, cols,
                                        d.nrows - r - 16 * part,
                                        [&](int j) { return __uint_as_float(v[16 * part + j]); });
                    }
                }
                if (!none) give_back();
            }
        }
        if (!ok && lane == 0) atomicOr(a.status, kStatusWaitTimeout);
    } else {
        if constexpr (kMoveRegisters) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const uint32_t full_at = PAIR ? map_to_cta(full, 0) : full;
        bool ok = true;
        if (warp == 0) {
            // Copies of whole blocks, and each stage's byte count.
            uint32_t it = 0;
            for (int t = first_tile; t < tiles && ok; t += tile_step) {
                const Tile d = tile_of<KIND, CTAS>(a, c, t);
                const int half = d.n / CTAS;               // B rows of this CTA
                const int b0 = d.row0 + rank * half;
                const int m0 = d.m0 + rank * 128;
                constexpr int kUnit = KIND == kWgrad ? 64 : GATHER ? 4 : 32;  // rows of a copy
                const uint32_t bytes = kABytes + round_up(half, kUnit) * kStep * 2;
                for (int s = 0; s < d.steps; ++s, ++it) {
                    const uint32_t stage = it % kStages, phase = it / kStages & 1;
                    // all lanes give up together: the warp meets again below
                    ok = __all_sync(0xffffffffu, mbar_wait_long<PAIR>(empty + 8 * stage, phase ^ 1,
                                                                     a.timeout_ns));
                    if (!ok) break;
                    const uint32_t bar = full_at + 8 * stage;
                    const uint32_t sa = base + stage * S::kStageBytes, sb = sa + kABytes;
                    const int c0 = s * kStep;
                    const bool whole = KIND != kWgrad || c0 + kStep <= d.summed;
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * stage, CTAS * bytes);
                        if (KIND == kForward) tma_3d<PAIR>(sa, &maps.a, c0, m0, d.expert, bar);
                        if (KIND == kDgrad)
                            for (int i = 0; i < 2; ++i)
                                tma_3d<PAIR>(sa + i * 8192, &maps.a, m0 + 64 * i, c0, d.expert, bar);
                        if (KIND != kWgrad && !GATHER)
                            for (int i = 0; i < half; i += 32)
                                tma_2d<PAIR>(sb + i * kStep * 2, &maps.b, c0, b0 + i, bar);
                        if (KIND == kWgrad && whole) {
                            const int r = d.sum0 + c0;
                            if (!GATHER)
                                for (int i = 0; i < 2; ++i)
                                    tma_2d<PAIR>(sa + i * 8192, &maps.a, m0 + 64 * i, r, bar);
                            for (int i = 0; i < half; i += 64)
                                tma_2d<PAIR>(sb + i / 64 * 8192, &maps.b, b0 + i, r, bar);
                        }
                        // the stage is free for warp 2's copies
                        if (KIND == kWgrad && !GATHER && !whole) mbar_arrive(tail + 8 * stage);
                    }
                    __syncwarp();
                }
            }
            // The products have read every stage (and in a pair, the other CTA's
            // completions have arrived here) before this CTA may leave.
            if (ok)
                for (uint32_t i = 0; i < kStages && i < it; ++i) {
                    const uint32_t p = it - 1 - i;
                    ok = ok && mbar_wait_long<PAIR>(empty + 8 * (p % kStages), p / kStages & 1,
                                                    a.timeout_ns);
                }
            if (!ok && rank == 0)  // the copies in flight, before the memory is given back
                for (uint32_t i = 0; i < kStages && i < it; ++i) {
                    const uint32_t p = it - 1 - i;
                    (void)mbar_wait_long<PAIR>(full + 8 * (p % kStages), p / kStages & 1,
                                               a.timeout_ns);
                }
        } else if (warp == 1 && rank == 0) {
            // Products.
            constexpr bool A_MN = KIND != kForward, B_MN = KIND == kWgrad;
            uint32_t it = 0, acc_n = 0;
            for (int t = first_tile; t < tiles && ok; t += tile_step) {
                const Tile d = tile_of<KIND, CTAS>(a, c, t);
                const uint32_t idesc = instr_desc(S::kM, d.n, A_MN, B_MN);
                for (int s = 0; s < d.steps; ++s, ++it) {
                    const int in_segment = SUMS ? s % kSegment : s;
                    if (in_segment == 0) {
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait_long<PAIR>(acc_empty + 8 * (acc_n & 1),
                                                             (acc_n >> 1 & 1) ^ 1, a.timeout_ns));
                        if (!ok) break;
                    }
                    const uint32_t stage = it % kStages;
                    ok = __all_sync(0xffffffffu, mbar_wait_long<PAIR>(full + 8 * stage,
                                                                     it / kStages & 1, a.timeout_ns));
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t sa = base + stage * S::kStageBytes, sb = sa + kABytes;
                    const uint32_t dst = tmem + (acc_n & 1) * kRowsMax;
                    // 16 summed values: 32 bytes along a K-major row, 16 rows of an MN-major
                    // block
                    const uint64_t da = smem_desc(sa, A_MN ? 8192 : 16, 1024);
                    const uint64_t db = smem_desc(sb, B_MN ? 8192 : 16, 1024);
                    const int parts = (min(kStep, d.summed - s * kStep) + 15) / 16;
                    const bool end = s + 1 == d.steps || (SUMS && in_segment == kSegment - 1);
                    if (elect_one()) {
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            if (p < parts)
                                mma_bf16<CTAS>(dst, da + p * ((A_MN ? 2048 : 32) >> 4),
                                               db + p * ((B_MN ? 2048 : 32) >> 4), idesc,
                                               in_segment + p > 0);
                        mma_commit<CTAS>(empty + 8 * stage);
                        if (end) mma_commit<CTAS>(acc_full + 8 * (acc_n & 1));
                    }
                    __syncwarp();
                    if (end) ++acc_n;
                }
            }
        } else if (GATHER && warp >= 2) {
            // Rows by number, four a copy (-1, no such row, arrives as zeros): rows of x
            // chosen by row_index, and the last rows of wgrad's dy.  One or two warps for
            // every stage: a warp issues one copy in some 80 cycles, and a stage takes 32 of
            // them in 512.  (A prefill of 32768 rows at 4096 x 4096: two warps for all stages
            // 1321 us, one per stage 751, two, reading the numbers eight at a time, 703; 16-byte
            // cp.async by one warp per stage 997, as the proxy fence waits for the copies.)  The numbers go through shared memory, so
            // that the elected lane reads them with uniform addresses.
            const int index = warp < 4 ? warp - 2 : warp - W::kFirstGather + 2;
            const uint32_t stage = index % kStages;
            const int sub = index / kStages;
            const uint32_t bar = full_at + 8 * stage;
            constexpr int kList = 256 / (kStages * W::kShare);
            int4 *list = c.list + index * kList;
            const uint32_t sa = base + stage * S::kStageBytes, sb = sa + kABytes;
            uint32_t it = sub < W::kShare ? stage : ~0u;  // this warp's next step, over the tiles
            uint32_t done = 0;                            // steps of the tiles before
            for (int t = first_tile; t < tiles && ok && it != ~0u; t += tile_step) {
                const Tile d = tile_of<KIND, CTAS>(a, c, t);
                const int half = d.n / CTAS;
                const int b0 = d.row0 + rank * half;
                const int m0 = d.m0 + rank * 128;
                const int row_end = KIND == kWgrad ? d.sum0 + d.summed : d.row0 + d.nrows;
                auto x_row = [&](int i) {
                    const int v = i < row_end ? __ldg(a.row_index + i) : -1;
                    return v >= 0 && v < a.x_rows ? v : -1;
                };
                if (KIND != kWgrad && it < done + d.steps) {
                    // every kShare-th four rows of the CTA's half
                    for (int q = lane; q < half / (4 * W::kShare); q += 32) {
                        const int i = b0 + 4 * (W::kShare * q + sub);
                        list[q] = make_int4(x_row(i), x_row(i + 1), x_row(i + 2), x_row(i + 3));
                    }
                    __syncwarp();
                }
                for (; it < done + d.steps; it += kStages) {
                    const int c0 = static_cast<int>(it - done) * kStep;
                    if (KIND == kWgrad) {
                        for (int i = lane; i < kStep; i += 32)
                            reinterpret_cast<int *>(list)[i] = x_row(d.sum0 + c0 + i);
                        __syncwarp();
                    }
                    ok = __all_sync(0xffffffffu, mbar_wait_long<PAIR>(empty + 8 * stage,
                                                           (it / kStages & 1) ^ 1, a.timeout_ns));
                    if (!ok) break;
                    if (elect_one()) {
                        // eight at a time: the numbers are read before the first copy
                        constexpr int kBatch = 8;
                        const int quads = KIND == kForward ? half / (4 * W::kShare) : kStep / 4;
                        for (int q0 = 0; q0 < quads; q0 += kBatch) {
                            int4 rows[kBatch];
#pragma unroll
                            for (int q = 0; q < kBatch; ++q)
                                if (q0 + q < quads) rows[q] = list[q0 + q];
#pragma unroll
                            for (int q = 0; q < kBatch; ++q) {
                                if (q0 + q >= quads) break;
                                if (KIND == kForward)
                                    tma_gather4<PAIR>(sb + (W::kShare * (q0 + q) + sub) * 512,
                                                      &maps.b4, c0, rows[q], bar);
                                else
#pragma unroll
                                    for (int h = 0; h < 2; h += W::kShare)
                                        tma_gather4<PAIR>(sa + (h + sub) * 8192 + (q0 + q) * 512,
                                                          &maps.a4, m0 + 64 * (h + sub), rows[q],
                                                          bar);
                            }
                        }
                        if (KIND == kWgrad) {
                            if (c0 + kStep > d.summed)
                                dy_tail<PAIR>(maps, sb, d.sum0 + c0, row_end, b0, half, sub,
                                              W::kShare, bar);
                        }
                    }
                    __syncwarp();
                }
                done += d.steps;
            }
        } else if (KIND == kWgrad && !GATHER && warp == 2) {
            // The step that holds a sum's last rows, by number.  Warp 0 says when its stage is
            // free: `empty` moves on at every step, whether this warp has seen it or not, and
            // a parity wait that is a phase late does not end.  A stage's `tail` cannot move
            // on without this warp: its next phase needs the stage again, which needs this
            // warp's copies.
            uint32_t it = 0;       // steps up to this tile's end
            uint32_t phases = 0;   // bit s: parity of stage s's next tail
            for (int t = first_tile; t < tiles; t += tile_step) {
                const Tile d = tile_of<KIND, CTAS>(a, c, t);
                it += d.steps;
                if (d.summed % kStep == 0) continue;
                const uint32_t stage = (it - 1) % kStages;
                ok = __all_sync(0xffffffffu, mbar_wait_long(tail + 8 * stage, phases >> stage & 1,
                                                       a.timeout_ns));
                if (!ok) break;
                phases ^= 1u << stage;
                const int half = d.n / CTAS;
                const int m0 = d.m0 + rank * 128;
                const int row_end = d.sum0 + d.summed;
                const uint32_t bar = full_at + 8 * stage;
                const uint32_t sa = base + stage * S::kStageBytes, sb = sa + kABytes;
                const int r0 = d.sum0 + (d.steps - 1) * kStep;
                if (elect_one()) {
                    for (int q = 0; q < kStep / 4; ++q)
                        for (int h = 0; h < 2; ++h)
                            tma_gather4<PAIR>(sa + h * 8192 + q * 512, &maps.a4, m0 + 64 * h,
                                              rows_until(r0 + 4 * q, row_end), bar);
                    dy_tail<PAIR>(maps, sb, r0, row_end, d.row0 + rank * half, half, 0, 1, bar);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) atomicOr(a.status, kStatusWaitTimeout);
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    if (PAIR) cluster_barrier();
    if (warp == 2) {
        tcgen05_fence_after();
        tmem_dealloc<CTAS>(tmem, kTmemColumns);
    }
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn g_encode = nullptr;  // the driver's encoder, found once (prepare)

// BF16 values, strides in elements, boxes of one step by `rows`.
bool encode(CUtensorMap *m, const void *p, int rank, const cuuint64_t (&sizes)[3],
            const int64_t (&strides)[2], int rows) {
    return encode_map(
        m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, rank, sizes,
        {static_cast<cuuint64_t>(strides[0]) * 2, static_cast<cuuint64_t>(strides[1]) * 2}, kStep,
        rows);
}

template <int KIND, int CTAS, bool GATHER, bool SUMS>
cudaError_t launch(const Maps &maps, const GroupedArgs &a, int64_t tiles, cudaStream_t s) {
    const unsigned ctas =
        static_cast<unsigned>(CTAS * min(tiles, int64_t{CTAS == 2 ? a.num_pairs : a.num_sms}));
    return launch_ex(grouped_gemm_kernel<KIND, CTAS, GATHER, SUMS>, dim3(ctas),
                     dim3(Warps<CTAS, SUMS, GATHER>::kThreads), kSmemBytes, s, CTAS, a.programmatic, maps,
                     a);
}

template <int CTAS, bool SUMS>
cudaError_t launch_ctas(const GroupedArgs &a, cudaStream_t s) {
    using u64 = cuuint64_t;
    constexpr int kM = 128 * CTAS;
    Maps m = {};
    const u64 n = a.n, k = a.k, E = a.num_experts, xr = a.x_rows, rows = a.rows;
    bool ok = true;
    if (a.kind != kWgrad)
        ok = encode(&m.a, a.w, 3, {k, n, E}, {a.w_ld, a.w_expert}, a.kind == kForward ? 128 : 64);
    if (a.kind == kForward) {
        ok = ok && encode(&m.b, a.x, 2, {k, xr, 1}, {a.x_ld, 0}, 32);
        ok = ok && encode(&m.b4, a.x, 2, {k, xr, 1}, {a.x_ld, 0}, 1);
    } else if (a.kind == kDgrad) {
        ok = ok && encode(&m.b, a.dy, 2, {n, rows, 1}, {a.dy_ld, 0}, 32);
    } else {
        ok = ok && encode(&m.a, a.x, 2, {k, xr, 1}, {a.x_ld, 0}, 64);
        ok = ok && encode(&m.a4, a.x, 2, {k, xr, 1}, {a.x_ld, 0}, 1);
        ok = ok && encode(&m.b, a.dy, 2, {n, rows, 1}, {a.dy_ld, 0}, 64);
        ok = ok && encode(&m.b4, a.dy, 2, {n, rows, 1}, {a.dy_ld, 0}, 1);
    }
    if (!ok) return cudaErrorInvalidValue;
    const int columns = a.kind == kForward ? a.n : a.k;
    const int64_t mt = (columns + kM - 1) / kM;
    // at most this many tiles: the experts' sizes are known on the device only
    const int64_t tiles = a.kind == kWgrad
                              ? mt * a.num_experts * ((a.n + kRowsMax - 1) / kRowsMax)
                              : mt * (a.rows / kRowsMax + min(int64_t{a.num_experts}, a.rows));
    // tiles are counted in 32 bits (results of so many do not fit into memory)
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    switch (a.kind) {
        case kForward:
            return a.row_index ? launch<kForward, CTAS, true, SUMS>(m, a, tiles, s)
                               : launch<kForward, CTAS, false, SUMS>(m, a, tiles, s);
        case kDgrad: return launch<kDgrad, CTAS, false, SUMS>(m, a, tiles, s);
        default:
            return a.row_index ? launch<kWgrad, CTAS, true, SUMS>(m, a, tiles, s)
                               : launch<kWgrad, CTAS, false, SUMS>(m, a, tiles, s);
    }
}

template <int CTAS, bool SUMS>
cudaError_t prepare_ctas() {
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e =
        cudaFuncSetAttribute(grouped_gemm_kernel<kForward, CTAS, false, SUMS>, attr, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grouped_gemm_kernel<kForward, CTAS, true, SUMS>, attr, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grouped_gemm_kernel<kDgrad, CTAS, false, SUMS>, attr, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grouped_gemm_kernel<kWgrad, CTAS, false, SUMS>, attr, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grouped_gemm_kernel<kWgrad, CTAS, true, SUMS>, attr, kSmemBytes);
    return e;
}

}  // namespace

bool encode_map(CUtensorMap *m, CUtensorMapDataType type, const void *p, int rank,
                const cuuint64_t (&sizes)[3], const cuuint64_t (&strides)[2], int columns,
                int rows) {
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(columns), static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return g_encode(m, type, rank, const_cast<void *>(p), sizes, strides, box, ones,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t find_encoder() {
    if (g_encode) return cudaSuccess;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeFn>(fn);
    return cudaSuccess;
}

cudaError_t prepare_grouped_gemm(int *pairs) {
    cudaError_t e = find_encoder();
    if (e == cudaSuccess) e = prepare_ctas<1, false>();
    if (e == cudaSuccess) e = prepare_ctas<1, true>();
    if (e == cudaSuccess) e = prepare_ctas<2, false>();
    if (e == cudaSuccess) e = prepare_ctas<2, true>();
    if (e != cudaSuccess) return e;
    // pairs of SMs that run at once: a persistent grid of more would leave some
    // pairs' tiles for a second wave
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(Warps<2, false, true>::kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(pairs, grouped_gemm_kernel<kForward, 2, true, false>, &cfg);
}

cudaError_t launch_grouped_gemm(const GroupedArgs &a, cudaStream_t s) {
    if (a.kind == kForward && few_rows(a.rows, a.num_experts)) return launch_grouped_rows(a, s);
    // Up to 128 columns single CTAs: half of a pair's tile would be empty (32768 rows of 4096
    // values: 128 columns 58.7 against 61.1 us, 64 columns 55.9 against 60.1; at 256 columns
    // 93 against 65).
    const bool narrow = (a.kind == kForward ? a.n : a.k) <= 128;
    const auto launch_sums = [&](const GroupedArgs &b) {
        return narrow ? launch_ctas<1, true>(b, s) : launch_ctas<2, true>(b, s);
    };
    const auto launch_one = [&](const GroupedArgs &b) {
        return narrow ? launch_ctas<1, false>(b, s) : launch_ctas<2, false>(b, s);
    };
    if (a.kind != kWgrad)
        return a.out_fp32 || (a.kind == kForward ? a.k : a.n) > kLongSum ? launch_sums(a)
                                                                         : launch_one(a);
    // The weights' gradient sums an expert's rows, whose number is known on the device only:
    // where there may be a long sum, a second launch takes those experts and the first leaves
    // them out (1.2 us where there are none; that kernel for all of them would cost more:
    // 16 experts of 2048 rows, 2048 x 4096: 333 us with FP32 results, 295 here).
    GroupedArgs part = a;
    part.sum_to = a.out_fp32 ? INT32_MAX : kLongSum;
    cudaError_t e = a.out_fp32 ? launch_sums(part) : launch_one(part);
    if (a.out_fp32 || a.rows <= kLongSum || e != cudaSuccess) return e;
    part.sum_from = kLongSum + 1;
    part.sum_to = INT32_MAX;
    return launch_sums(part);
}

}  // namespace mf
