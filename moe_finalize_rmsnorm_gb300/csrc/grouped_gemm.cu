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
// tile may be any multiple of 16 up to 256: an expert of 40 rows costs 48, not
// 128 or 256.  An expert's rows are split evenly over its tiles.  In wgrad the
// ragged dimension is the summed one; the step that holds an expert's last rows
// reads them by number, and the rows behind them as zeros, so that a row of
// another expert (or one that was never written) enters nothing.
//
// One persistent CTA (or pair of CTAs: one tile of 256 columns over two SMs,
// each holding half of either operand) per SM walks the tiles: a warp that
// issues the copies of blocks (TMA, 128-byte swizzle, 64 summed values a step), a
// warp that issues the products into one of two accumulators in TMEM, four warps
// that move the other accumulator out, and one more per stage for rows that are gathered.
#include "experts.cuh"
#include "experts.h"
#include "tensor_map.h"

namespace mf {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsMax = 256;               // N of a tile
constexpr int kStep = 64;                   // summed values per stage: 128 bytes of BF16
constexpr int kABytes = 128 * kStep * 2;    // A of one CTA and stage
constexpr int kEpilogueBytes = 4 * 32 * 128;  // one 32 x 32 FP32 block per warp
constexpr int kTmemColumns = 512;           // two accumulators of 256

template <int CTAS>
struct Shape {
    static constexpr int kBBytes = kRowsMax / CTAS * kStep * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = CTAS == 2 ? 6 : 4;  // 192 KB either way
    static constexpr int kM = 128 * CTAS;
    static constexpr int kGatherThreads = kThreads + 32 * kStages;  // a warp per stage
};

// Shared memory behind the stages and the epilogue's blocks.
struct Control {
    int4 list[256];              // rows by number, four a copy; a part for each stage
    uint64_t full[6], empty[6], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int scan[8];
    int tiles[kMaxExperts + 1];  // row tiles of the experts before this one
    int lo[kMaxExperts + 1];     // first row; the next expert's is the end
};

constexpr int kSmemBytes = 1024 + 192 * 1024 + kEpilogueBytes + sizeof(Control);
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

template <int KIND, int CTAS>
__device__ __forceinline__ Tile tile_of(const GroupedArgs &a, const Control &c, int64_t t) {
    constexpr int M = Shape<CTAS>::kM;
    const int columns = KIND == kForward ? a.n : a.k;
    const int mt = (columns + M - 1) / M;
    Tile r;
    if (KIND == kWgrad) {
        const int nt = (a.n + kRowsMax - 1) / kRowsMax;
        r.expert = static_cast<int>(t / (int64_t{mt} * nt));
        const int local = static_cast<int>(t - r.expert * (int64_t{mt} * nt));
        r.m0 = local % mt * M;
        r.row0 = local / mt * kRowsMax;
        r.nrows = min(kRowsMax, a.n - r.row0);
        r.summed = max(c.lo[r.expert + 1] - c.lo[r.expert], 0);
        r.sum0 = c.lo[r.expert];
    } else {
        const int u = static_cast<int>(t / mt);
        int e = 0;  // the last expert whose tiles start at or before u
        for (int step = 512; step > 0; step /= 2)
            if (e + step < a.num_experts && c.tiles[e + step] <= u) e += step;
        r.expert = e;
        const int rows = c.lo[e + 1] - c.lo[e];
        const int rt = c.tiles[e + 1] - c.tiles[e];
        const int local = static_cast<int>(t - c.tiles[e] * int64_t{mt});
        const int each = round_up((rows + rt - 1) / rt, 16);
        const int first = min(local % rt * each, rows);
        r.m0 = local / rt * M;
        r.row0 = c.lo[e] + first;
        r.nrows = min(each, rows - first);
        r.summed = KIND == kForward ? a.k : a.n;
        r.sum0 = 0;
    }
    r.n = round_up(r.nrows, 16 * CTAS);
    r.steps = (r.summed + kStep - 1) / kStep;
    return r;
}

template <int KIND, int CTAS, bool GATHER>
__global__ void __launch_bounds__(GATHER ? Shape<CTAS>::kGatherThreads : kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ Maps maps, const GroupedArgs a) {
    using S = Shape<CTAS>;
    constexpr bool PAIR = CTAS == 2;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t *aligned_raw = raw + (base - smem_u32(raw));
    uint8_t *blocks = aligned_raw + S::kStages * S::kStageBytes;
    Control &c = *reinterpret_cast<Control *>(blocks + kEpilogueBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const uint32_t full = smem_u32(c.full), empty = smem_u32(c.empty);
    const uint32_t acc_full = smem_u32(c.acc_full), acc_empty = smem_u32(c.acc_empty);

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 4 * CTAS);
        }
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc<CTAS>(smem_u32(&c.tmem), kTmemColumns);

    // The experts' rows and their tiles' numbers (an exclusive scan, each thread
    // a run of experts).
    pdl_wait();
    const int per = (a.num_experts + kThreads - 1) / kThreads;
    const int first = min(static_cast<int>(threadIdx.x) * per, a.num_experts);
    const int last = min(first + per, a.num_experts);
    int sum = 0;
    for (int e = first; e < last; ++e) {
        int lo, hi;
        expert_rows(a.offsets, e, static_cast<int>(a.rows), lo, hi);
        c.lo[e] = lo;
        if (e + 1 == a.num_experts) c.lo[e + 1] = hi;
        c.tiles[e] = sum;
        sum += (hi - lo + kRowsMax - 1) / kRowsMax;
    }
    int before = sum;
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31 && warp < 8) c.scan[warp] = before;
    before -= sum;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += c.scan[w];
        total += c.scan[w];
    }
    for (int e = first; e < last; ++e) c.tiles[e] += before;
    if (threadIdx.x == 0) c.tiles[a.num_experts] = total;
    tcgen05_fence_before();
    __syncthreads();
    if (PAIR) cluster_barrier();
    tcgen05_fence_after();
    const uint32_t tmem = c.tmem;

    const int columns = KIND == kForward ? a.n : a.k;
    const int64_t mt = (columns + S::kM - 1) / S::kM;
    const int64_t tiles = KIND == kWgrad
                              ? int64_t{a.num_experts} * mt * ((a.n + kRowsMax - 1) / kRowsMax)
                              : mt * total;
    const int64_t first_tile = blockIdx.x / CTAS, tile_step = gridDim.x / CTAS;

    if (warp == 0) {
        // Copies of whole blocks, and each stage's byte count.
        const uint32_t full_at = PAIR ? map_to_cta(full, 0) : full;
        uint32_t it = 0;
        bool ok = true;
        for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
            const Tile d = tile_of<KIND, CTAS>(a, c, t);
            const int half = d.n / CTAS;               // B rows of this CTA
            const int b0 = d.row0 + rank * half;
            const int m0 = d.m0 + rank * 128;
            const uint32_t a_bytes = kABytes;
            const uint32_t b_bytes = KIND == kWgrad ? round_up(half, 64) * kStep * 2
                                     : GATHER       ? half * kStep * 2
                                                    : round_up(half, 32) * kStep * 2;
            for (int s = 0; s < d.steps; ++s, ++it) {
                const uint32_t stage = it % S::kStages, phase = it / S::kStages & 1;
                // all lanes give up together: the warp meets again below
                ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * stage, phase ^ 1, a.timeout_ns));
                if (!ok) break;
                const uint32_t bar = full_at + 8 * stage;
                const uint32_t sa = base + stage * S::kStageBytes, sb = sa + kABytes;
                const int c0 = s * kStep;
                const bool whole = KIND != kWgrad || c0 + kStep <= d.summed;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * stage, CTAS * (a_bytes + b_bytes));
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
                }
                __syncwarp();
            }
        }
        // The products have read every stage (and in a pair, the other CTA's
        // completions have arrived here) before this CTA may leave.
        if (ok)
            for (uint32_t i = 0; i < S::kStages && i < it; ++i) {
                const uint32_t p = it - 1 - i;
                ok = ok && mbar_wait(empty + 8 * (p % S::kStages), p / S::kStages & 1,
                                     a.timeout_ns);
            }
        if (!ok) {
            if (lane == 0) atomicOr(a.status, kStatusWaitTimeout);
            if (rank == 0)  // the copies in flight, before the memory is given back
                for (uint32_t i = 0; i < S::kStages && i < it; ++i) {
                    const uint32_t p = it - 1 - i;
                    (void)mbar_wait(full + 8 * (p % S::kStages), p / S::kStages & 1, a.timeout_ns);
                }
        }
    } else if (KIND == kWgrad && warp == 2) {
        // Copies of rows by number (four a copy), only for the step that holds a
        // sum's last rows: -1 behind them arrives as zeros.
        const uint32_t full_at = PAIR ? map_to_cta(full, 0) : full;
        uint32_t it = 0;
        bool ok = true;
        for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
            const Tile d = tile_of<KIND, CTAS>(a, c, t);
            const int half = d.n / CTAS;
            const int b0 = d.row0 + rank * half;
            const int m0 = d.m0 + rank * 128;
            const int row_end = d.sum0 + d.summed;
            for (int s = 0; s < d.steps; ++s, ++it) {
                const uint32_t stage = it % S::kStages, phase = it / S::kStages & 1;
                const int c0 = s * kStep;
                ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * stage, phase ^ 1, a.timeout_ns));
                if (!ok) break;
                const uint32_t bar = full_at + 8 * stage;
                const uint32_t sa = base + stage * S::kStageBytes, sb = sa + kABytes;
                if (c0 + kStep > d.summed && elect_one()) {
                    auto row = [&](int i) { return i < row_end ? i : -1; };
                    for (int q = 0; q < kStep / 4; ++q) {
                        const int i = d.sum0 + c0 + 4 * q;
                        const int4 rows = make_int4(row(i), row(i + 1), row(i + 2), row(i + 3));
                        if (!GATHER)
                            for (int h = 0; h < 2; ++h)
                                tma_gather4<PAIR>(sa + h * 8192 + q * 512, &maps.a4, m0 + 64 * h,
                                                  rows, bar);
                        for (int at = 0; at < half; at += 64)
                            tma_gather4<PAIR>(sb + at / 64 * 8192 + q * 512, &maps.b4, b0 + at, rows,
                                              bar);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) atomicOr(a.status, kStatusWaitTimeout);
    } else if (GATHER && warp >= 8) {
        // Rows of x chosen by row_index, four a copy (-1, no such row, arrives as
        // zeros), one warp per stage: a warp issues one copy in some 80 cycles, and a
        // stage takes 32 of them in 512.  Two warps for all stages: 1321 us for a
        // prefill of 32768 rows at 4096 x 4096, one per stage: 751; 16-byte cp.async by
        // one warp per stage: 997 (the proxy fence waits for the copies).
        // The numbers go through shared memory, so that the elected lane reads them with
        // uniform addresses.
        const uint32_t stage = warp - 8;
        const uint32_t bar = (PAIR ? map_to_cta(full, 0) : full) + 8 * stage;
        int4 *list = c.list + stage * (64 / CTAS);
        const uint32_t dst = base + stage * S::kStageBytes + (KIND == kWgrad ? 0 : kABytes);
        uint32_t it = stage;   // this warp's next step, counted over the tiles
        uint32_t done = 0;     // steps of the tiles before
        bool ok = true;
        for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
            const Tile d = tile_of<KIND, CTAS>(a, c, t);
            const int half = d.n / CTAS;
            const int row_end = KIND == kWgrad ? d.sum0 + d.summed : d.row0 + d.nrows;
            const int m0 = d.m0 + rank * 128;
            auto x_row = [&](int i) {
                const int v = i < row_end ? __ldg(a.row_index + i) : -1;
                return v >= 0 && v < a.x_rows ? v : -1;
            };
            if (KIND != kWgrad && it < done + d.steps) {
                for (int i = lane; i < half; i += 32)
                    reinterpret_cast<int *>(list)[i] = x_row(d.row0 + rank * half + i);
                __syncwarp();
            }
            for (; it < done + d.steps; it += S::kStages) {
                const int c0 = static_cast<int>(it - done) * kStep;
                if (KIND == kWgrad) {
                    for (int i = lane; i < 64; i += 32)
                        reinterpret_cast<int *>(list)[i] = x_row(d.sum0 + c0 + i);
                    __syncwarp();
                }
                ok = __all_sync(0xffffffffu,
                                mbar_wait(empty + 8 * stage, (it / S::kStages & 1) ^ 1, a.timeout_ns));
                if (!ok) break;
                if (elect_one()) {
                    if (KIND == kForward) {
#pragma unroll 8
                        for (int q = 0; q < half / 4; ++q)
                            tma_gather4<PAIR>(dst + q * 512, &maps.b4, c0, list[q], bar);
                    } else {
#pragma unroll 8
                        for (int q = 0; q < 16; ++q) {
                            const int4 r = list[q];
                            tma_gather4<PAIR>(dst + q * 512, &maps.a4, m0, r, bar);
                            tma_gather4<PAIR>(dst + 8192 + q * 512, &maps.a4, m0 + 64, r, bar);
                        }
                    }
                }
                __syncwarp();
            }
            done += d.steps;
        }
        if (!ok && lane == 0) atomicOr(a.status, kStatusWaitTimeout);
    } else if (warp == 1 && rank == 0) {
        // Products.
        constexpr bool A_MN = KIND != kForward, B_MN = KIND == kWgrad;
        uint32_t it = 0, acc = 0;
        bool ok = true;
        for (int64_t t = first_tile; t < tiles && ok; t += tile_step) {
            const Tile d = tile_of<KIND, CTAS>(a, c, t);
            if (d.steps == 0) continue;
            ok = __all_sync(0xffffffffu, mbar_wait(acc_empty + 8 * (acc & 1), (acc >> 1 & 1) ^ 1,
                                                   a.timeout_ns));
            if (!ok) break;
            tcgen05_fence_after();
            const uint32_t idesc = instr_desc(S::kM, d.n, A_MN, B_MN);
            const uint32_t dst = tmem + (acc & 1) * kRowsMax;
            for (int s = 0; s < d.steps; ++s, ++it) {
                const uint32_t stage = it % S::kStages;
                ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * stage, it / S::kStages & 1,
                                                       a.timeout_ns));
                if (!ok) break;
                tcgen05_fence_after();
                const uint32_t sa = base + stage * S::kStageBytes, sb = sa + kABytes;
                // 16 summed values: 32 bytes along a K-major row, 16 rows of an MN-major block
                const uint64_t da = smem_desc(sa, A_MN ? 8192 : 16, 1024);
                const uint64_t db = smem_desc(sb, B_MN ? 8192 : 16, 1024);
                const int parts = (min(kStep, d.summed - s * kStep) + 15) / 16;
                if (elect_one()) {
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        if (p < parts)
                            mma_bf16<CTAS>(dst, da + p * ((A_MN ? 2048 : 32) >> 4),
                                           db + p * ((B_MN ? 2048 : 32) >> 4), idesc, s + p > 0);
                    mma_commit<CTAS>(empty + 8 * stage);
                    if (s + 1 == d.steps) mma_commit<CTAS>(acc_full + 8 * (acc & 1));
                }
                __syncwarp();
            }
            ++acc;
        }
        if (!ok && lane == 0) atomicOr(a.status, kStatusWaitTimeout);
    } else if (warp >= 4 && warp < 8) {
        // Results: lane = output column, register = output row.  Each warp turns
        // its 32 x 32 block in shared memory and stores 64 (BF16) or 128 bytes of
        // every row.
        const int w = warp - 4;
        uint8_t *block = blocks + w * 32 * 128;
        const uint32_t done_at = PAIR ? map_to_cta(acc_empty, 0) : acc_empty;
        uint32_t acc = 0;
        bool ok = true;
        for (int64_t t = first_tile; t < tiles; t += tile_step) {
            const Tile d = tile_of<KIND, CTAS>(a, c, t);
            const bool empty_sum = d.steps == 0;
            if (empty_sum && (a.accumulate || d.nrows == 0)) continue;
            if (!empty_sum) {
                ok = __all_sync(0xffffffffu, mbar_wait(acc_full + 8 * (acc & 1), acc >> 1 & 1,
                                                       a.timeout_ns));
                if (!ok) break;
                tcgen05_fence_after();
            }
            const int col0 = d.m0 + rank * 128 + w * 32;
            const int64_t ld = KIND == kWgrad ? a.k : a.out_ld;
            const int64_t out0 =
                (KIND == kWgrad ? int64_t{d.expert} * a.n + d.row0 : int64_t{d.row0}) * ld + col0;
            for (int r0 = 0; r0 < d.nrows; r0 += 32) {
                uint32_t v[32];
                if (empty_sum) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0;
                } else {
                    tmem_ld32(tmem + (acc & 1) * kRowsMax + r0 + (static_cast<uint32_t>(w * 32) << 16),
                              v);
                }
                if (a.out_fp32) {
                    float *f = reinterpret_cast<float *>(block);
#pragma unroll
                    for (int j = 0; j < 32; ++j) f[j * 32 + lane] = __uint_as_float(v[j]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = i * 4 + lane / 8, col = lane % 8 * 4;
                        if (r0 + r < d.nrows && col0 + col < columns) {
                            float4 x = *reinterpret_cast<float4 *>(f + r * 32 + col);
                            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) +
                                                                   out0 + (r0 + r) * ld + col);
                            if (KIND == kWgrad && a.accumulate) {
                                const float4 y = *o;
                                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                            }
                            *o = x;
                        }
                    }
                } else {
                    __nv_bfloat16 *h = reinterpret_cast<__nv_bfloat16 *>(block);
                    const bool add = KIND == kWgrad && a.accumulate;
                    if (!add) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            h[j * 32 + lane] = __float2bfloat16_rn(__uint_as_float(v[j]));
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = i * 8 + lane / 4, col = lane % 4 * 8;
                            if (r0 + r < d.nrows && col0 + col < columns)
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                           out0 + (r0 + r) * ld + col) =
                                    *reinterpret_cast<uint4 *>(h + r * 32 + col);
                        }
                    } else {
                        // the sum with what the output holds is rounded once
                        float *f = reinterpret_cast<float *>(block);
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j * 32 + lane] = __uint_as_float(v[j]);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = i * 8 + lane / 4, col = lane % 4 * 8;
                            if (r0 + r < d.nrows && col0 + col < columns) {
                                uint4 *o = reinterpret_cast<uint4 *>(
                                    static_cast<__nv_bfloat16 *>(a.out) + out0 + (r0 + r) * ld + col);
                                float y[8];
                                unpack8(*o, y);
#pragma unroll
                                for (int u = 0; u < 8; ++u) y[u] += f[r * 32 + col + u];
                                *o = pack8_rn(y);
                            }
                        }
                    }
                }
                __syncwarp();
            }
            if (!empty_sum) {
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(done_at + 8 * (acc & 1));
                ++acc;
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

template <int KIND, int CTAS, bool GATHER>
cudaError_t launch(const Maps &maps, const GroupedArgs &a, int64_t tiles, cudaStream_t s) {
    const unsigned ctas =
        static_cast<unsigned>(CTAS * min(tiles, int64_t{CTAS == 2 ? a.num_pairs : a.num_sms}));
    return launch_ex(grouped_gemm_kernel<KIND, CTAS, GATHER>, dim3(ctas),
                     dim3(GATHER ? Shape<CTAS>::kGatherThreads : kThreads), kSmemBytes, s, CTAS, a.programmatic, maps, a);
}

template <int CTAS>
cudaError_t launch_ctas(const GroupedArgs &a, cudaStream_t s) {
    using u64 = cuuint64_t;
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
    const int64_t mt = (columns + Shape<CTAS>::kM - 1) / Shape<CTAS>::kM;
    // at most this many tiles: the experts' sizes are known on the device only
    const int64_t tiles =
        a.kind == kWgrad
            ? mt * a.num_experts * ((a.n + kRowsMax - 1) / kRowsMax)
            : mt * (a.rows / kRowsMax + min(int64_t{a.num_experts}, a.rows));
    switch (a.kind) {
        case kForward:
            return a.row_index ? launch<kForward, CTAS, true>(m, a, tiles, s)
                               : launch<kForward, CTAS, false>(m, a, tiles, s);
        case kDgrad: return launch<kDgrad, CTAS, false>(m, a, tiles, s);
        default:
            return a.row_index ? launch<kWgrad, CTAS, true>(m, a, tiles, s)
                               : launch<kWgrad, CTAS, false>(m, a, tiles, s);
    }
}

template <int CTAS>
cudaError_t prepare_ctas() {
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(grouped_gemm_kernel<kForward, CTAS, false>, attr, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grouped_gemm_kernel<kForward, CTAS, true>, attr, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grouped_gemm_kernel<kDgrad, CTAS, false>, attr, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grouped_gemm_kernel<kWgrad, CTAS, false>, attr, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grouped_gemm_kernel<kWgrad, CTAS, true>, attr, kSmemBytes);
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

cudaError_t prepare_grouped_gemm(int *pairs) {
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                         cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        g_encode = reinterpret_cast<EncodeFn>(fn);
    }
    cudaError_t e = prepare_ctas<1>();
    if (e == cudaSuccess) e = prepare_ctas<2>();
    if (e != cudaSuccess) return e;
    // pairs of SMs that run at once: a persistent grid of more would leave some
    // pairs' tiles for a second wave
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(pairs, grouped_gemm_kernel<kForward, 2, false>, &cfg);
}

cudaError_t launch_grouped_gemm(const GroupedArgs &a, cudaStream_t s) {
    return (a.kind == kForward ? a.n : a.k) <= 128 ? launch_ctas<1>(a, s) : launch_ctas<2>(a, s);
}

}  // namespace mf
