// Products of few rows per expert with 4-bit weights and group scales.
//
// Bound by the weights' bytes: each is read once for every 8, 16 or 32 rows of its
// expert.  A warp takes 32 columns n and up to so many rows.  It streams 256 summed
// values of its 32 columns a stage (128 bytes a column) through its own ring in
// shared memory, one tensor-map copy a stage, turns the nibbles into (q - z) / 64 in
// BF16 (exact), and multiplies with the rows in mma.m16n8k16, n along M, the rows
// along N: with so few rows the tensor cores only have to keep up with the
// conversion.  Each group's FP32 sum is scaled once (and by 64 at the end).  Warps
// that share a column block split the summed values between them and add up through
// shared memory, in warp order.
//
// Measured (GB300, device time): one token through eight 4096 x 4096 matrices, groups of
// 128, 18.3 us (69 MB; 10.2 at the copy bandwidth, some 4 of start); eight tokens through
// 41 of them 75 us (4.9 TB/s); 512 rows through 64 matrices of 4096 x 2048, groups of 32
// with zeros, 100 us (3.2 TB/s).  What bounds it is the issue of instructions: 71 to 106 for
// 1024 weights, of which 36 convert them.  Summed values that are no whole stages (k not a
// multiple of 256) take the forms without WHOLE, which load scales word by word and, with
// passes of 16 and 32 rows, keep up to 488 bytes a thread in local memory: k = 2880 152 us
// where 2816 takes 109 (512 rows, 64 experts, groups of 32), 24 and 17 (64 rows, 8
// experts), 15.7 and 14.0 (8 rows).
#include "experts.h"
#include "few_rows.cuh"
#include "tensor_map.h"

namespace mf {
namespace {

// Warps of a CTA: for passes of 32 rows 12, with the registers of 16.
constexpr int warps_of(int tiles) { return tiles == 4 ? 12 : 16; }
constexpr int kCols = 32;      // n of a warp
constexpr int kSpan = 256;     // summed values of a stage: 128 bytes of a column
constexpr int kStages = 2;
constexpr int kWeightBytes = kCols * kSpan / 2;

// A stage's scales and zeros per column: FP32, or the words that hold the BF16 from
// either half of a word on, or the bytes from any byte on.
template <int GROUP>
struct GroupData {
    static constexpr int kGroups = kSpan / GROUP;
    static constexpr int kScalePitch = 4 * kGroups;
    static constexpr int kZeroPitch = kGroups == 8 ? 16 : 8;
    static constexpr int kZeroAt = kCols * kScalePitch;
    static constexpr int kBytes = kZeroAt + kCols * kZeroPitch;
};

struct GemvControl {
    uint64_t full[16][kStages];
    int scan[16];
    int tiles[kMaxExperts + 1];  // passes of the experts before this one
    int lo[kMaxExperts + 1];     // first row
};

// One CTA: the stages, the partial results of 8 TILES rows for every warp, the control.
template <int GROUP, int TILES>
struct GemvSmem {
    static constexpr int kSumBytes = kCols * 8 * TILES * 4;
    static constexpr int kBytes =
        1024 + warps_of(TILES) * (kStages * (kWeightBytes + GroupData<GROUP>::kBytes) + kSumBytes) +
        static_cast<int>(sizeof(GemvControl));
    static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
};

// 4, 8 or 16 bytes global -> shared.
template <int BYTES>
__device__ __forceinline__ void cp_async_ca(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}

// 4 bytes global -> shared, the bytes behind `bytes` (0..4) as zeros.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

// a * b + c on two BF16, one rounding.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// c += a * b on two FP32.
__device__ __forceinline__ void fma_f32x2(float &c0, float &c1, float a, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "mov.b64 c, {%0, %1};\n\tfma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(c0), "+f"(c1)
        : "f"(a), "f"(b0), "f"(b1));
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&v)[N]) {
    if constexpr (N == 1) {
        v[0] = lds<uint32_t>(addr);
    } else if constexpr (N == 2) {
        const uint2 q = lds<uint2>(addr);
        v[0] = q.x;
        v[1] = q.y;
    } else {
        static_assert(N == 4, "");
        const uint4 q = lds<uint4>(addr);
        v[0] = q.x;
        v[1] = q.y;
        v[2] = q.z;
        v[3] = q.w;
    }
}

// The same for the copies.
struct Copies {
    int item;
    int stage;
    int expert, n0;
    int64_t o;  // number of the first scale of the lane's column in this stage
};

// TILES: a pass takes up to 8 TILES rows.  WHOLE: the summed values are whole
// stages, so that a stage's scales are aligned to their size (and its zeros, where
// a group is at most 64 long).
template <int GROUP, int TILES, bool WHOLE>
struct Gemv {
    using G = GroupData<GROUP>;
    static constexpr int kGroups = G::kGroups;
    static constexpr int kRowsPass = 8 * TILES;
    static constexpr bool kWholeZeros = WHOLE && kGroups >= 4;

    const GemvArgs &a;
    const CUtensorMap &map;
    const GemvControl &c;
    const int lane, g, t;
    const int share, part;  // warps of a column block, this one's number
    const int step, items;
    const unsigned col_blocks;
    const int spans, groups;
    const int search;           // first step of the search for an expert
    const uint32_t weights_at, group_at, full;  // this warp's stages and barriers
    float *sums;  // of the block's first warp
    const int barrier;

    __device__ int expert_of(int pass) const {
        return expert_of_pass(c.tiles, a.num_experts, search, pass);
    }

    __device__ void locate(Cursor &p) const {
        if (p.item >= items) return;
        const int pass = p.item / col_blocks;
        p.expert = expert_of(pass);
        p.n0 = (p.item - pass * col_blocks) * kCols;
        const int first_row = (pass - c.tiles[p.expert]) * kRowsPass;
        p.row0 = c.lo[p.expert] + first_row;
        p.rows = min(kRowsPass, c.lo[p.expert + 1] - p.row0);
    }

    __device__ void locate(Copies &p) const {
        if (p.item >= items) return;
        const int pass = p.item / col_blocks;
        p.expert = expert_of(pass);
        p.n0 = (p.item - pass * col_blocks) * kCols;
        // columns behind the last stand for it: their results are not stored
        p.o = (int64_t{p.expert} * a.n + min(p.n0 + lane, a.n - 1)) * groups + part * kGroups;
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
            if (elect_one()) {
                mbar_arrive_expect_tx(full + 8 * slot, kWeightBytes);
                tma_3d<false>(weights_at + slot * kWeightBytes, &map, p.stage * (kSpan / 2), p.n0,
                              p.expert, full + 8 * slot);
            }
            __syncwarp();
            const int ng = WHOLE ? kGroups : min(kGroups, groups - p.stage * kGroups);
            const uint32_t sd = group_at + slot * G::kBytes + lane * G::kScalePitch;
            const uint32_t zd = group_at + slot * G::kBytes + G::kZeroAt + lane * G::kZeroPitch;
            if (a.scale_fp32) {
                const float *s = static_cast<const float *>(a.scales) + p.o;
                if constexpr (WHOLE) {
                    constexpr int kBytes = kGroups == 2 ? 8 : 16;
#pragma unroll
                    for (int i = 0; i < 4 * kGroups / kBytes; ++i)
                        cp_async_ca<kBytes>(sd + kBytes * i, s + kBytes / 4 * i);
                } else {
#pragma unroll
                    for (int i = 0; i < kGroups; ++i)
                        if (i < ng) cp_async_4(sd + 4 * i, s + i, 4);
                }
            } else if constexpr (WHOLE) {
                cp_async_ca<2 * kGroups>(sd, static_cast<const uint16_t *>(a.scales) + p.o);
            } else {
                // the aligned words that hold the scales
                const uint8_t *s = static_cast<const uint8_t *>(a.scales) + (p.o & ~int64_t{1}) * 2;
                const int bytes = (static_cast<int>(p.o & 1) + ng) * 2;
#pragma unroll
                for (int i = 0; i < kGroups / 2 + 1; ++i)
                    if (4 * i < bytes) cp_async_4(sd + 4 * i, s + 4 * i, min(4, bytes - 4 * i));
            }
            if (a.zeros) {
                if constexpr (kWholeZeros) {
                    cp_async_ca<kGroups>(zd, a.zeros + p.o);
                } else {
                    const uint8_t *z = a.zeros + (p.o & ~int64_t{3});
                    const int bytes = static_cast<int>(p.o & 3) + ng;
#pragma unroll
                    for (int i = 0; i < (kGroups + 6) / 4; ++i)
                        if (4 * i < bytes) cp_async_4(zd + 4 * i, z + 4 * i, min(4, bytes - 4 * i));
                }
            }
            p.stage += share;
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
        const int64_t at = (int64_t{d.row0} + r) * a.out_ld + d.n0 + n;
        if (a.out_fp32)
            static_cast<float *>(a.out)[at] = v;
        else
            static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
    }

    // One column block with up to 8 NT rows.  A copy that does not arrive within
    // `limit` sets the status and the limit to zero: the warp goes on (the others
    // wait for it at the block's barrier), with results of no meaning.
    template <int NT>
    __device__ void item(Cursor &now, Copies &ahead, uint32_t &it, uint64_t &limit) const {
        const Cursor d = now;
        // The rows this thread feeds (row g of every eight).  Where there is none, any
        // row will do: its results are not stored, or stored as zeros.
        const __nv_bfloat16 *x[NT];
        unsigned outside[NT];  // bit 4 j: row j of every eight is not in x
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int row = x_row(d, min(8 * i + g, d.rows - 1));
            outside[i] = __ballot_sync(0xffffffffu, row < 0);
            x[i] = static_cast<const __nv_bfloat16 *>(a.x) + max(row, 0) * a.x_ld + 8 * t +
                   now.stage * kSpan;
        }
        // The rows' values of the next kAhead blocks of 32, loaded that long before they
        // are used: they come from the L2, some 800 cycles away.
        constexpr int kAhead = 4 / NT;
        uint4 xv[kAhead][NT];
        auto load_x = [&](int b, int k) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                xv[b % kAhead][i] = __ldg(reinterpret_cast<const uint4 *>(x[i] + k + 32 * b));
        };
        {
            const int blocks = WHOLE ? 8 : min(kSpan, a.k - now.stage * kSpan) / 32;
#pragma unroll
            for (int b = 0; b < kAhead; ++b)
                if (b < blocks) load_x(b, 0);
        }
        // Number of the first scale of column g (those of columns g + 8 i differ by
        // multiples of 8): modulo 2 and 4 it says where the copied words hold the scales
        // and the zeros.  A stage moves it by an even number.
        const unsigned skip = static_cast<unsigned>((int64_t{d.expert} * a.n + d.n0 + g) * groups);
        float acc[2][NT][4] = {};
        while (now.item == d.item) {
            const int blocks = WHOLE ? 8 : min(kSpan, a.k - now.stage * kSpan) / 32;
            const uint32_t slot = it % kStages;
            cp_async_wait<kStages - 2>();
            __syncwarp();  // the other lanes' copies too
            if (limit == 0 ||
                !__all_sync(0xffffffffu, mbar_wait_long(full + 8 * slot, it / kStages & 1, limit))) {
                limit = 0;
                if (lane == 0) atomicOr(a.status, kStatusWaitTimeout);
            }
            issue(ahead, (it + kStages - 1) % kStages);
            const uint32_t wd = weights_at + slot * kWeightBytes + g * 128 + t * 4 + (g << 4);
            const uint32_t gd = group_at + slot * G::kBytes;
            const uint32_t sd =
                gd + g * G::kScalePitch + (WHOLE || a.scale_fp32 ? 0 : (skip & 1u) * 2);
            const uint32_t zd = gd + G::kZeroAt + g * G::kZeroPitch +
                                (kWholeZeros ? 0 : (skip + now.stage * kGroups) & 3u);
            advance(now);
            // blocks of the item's next stage
            const int next = now.item != d.item ? 0
                             : WHOLE            ? 8
                                                : min(kSpan, a.k - now.stage * kSpan) / 32;
            // written out twice where the registers allow it (73 against 78 us, 8 tokens)
            constexpr int kUnroll = TILES == 1 ? 2 : 1;
#pragma unroll kUnroll
            for (int half = 0; half < 2; ++half) {
                const int left = WHOLE ? 4 : blocks - 4 * half;  // blocks from here on
                const int after = half ? next : blocks - 4;
                // the scales and zeros of the half's groups, as they lie in memory
                constexpr int kHere = kGroups / 2;
                constexpr int kPer = GROUP / 32;  // blocks of a group
                uint32_t sv[4][kHere], zv[4];
                if constexpr (WHOLE) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t at = sd + 8 * i * G::kScalePitch;
                        if (a.scale_fp32) {
                            lds_words<kHere>(at + 4 * kHere * half, sv[i]);
                        } else if constexpr (kHere == 1) {
                            sv[i][0] = uint32_t{lds<uint16_t>(at + 2 * half)} << 16;
                        } else {
                            uint32_t two[kHere / 2];
                            lds_words<kHere / 2>(at + 2 * kHere * half, two);
#pragma unroll
                            for (int j = 0; j < kHere; ++j)
                                sv[i][j] = j & 1 ? two[j / 2] & 0xFFFF0000u : two[j / 2] << 16;
                        }
                    }
                }
                if (kWholeZeros && a.zeros) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t at = zd + 8 * i * G::kZeroPitch + kHere * half;
                        if constexpr (kHere == 4)
                            zv[i] = lds<uint32_t>(at);
                        else
                            zv[i] = lds<uint16_t>(at);
                    }
                }
                const int x_next = half ? share * kSpan - 128 : 128;
                const uint32_t wh = wd ^ half << 6;
                float sum[2][NT][4];
                uint32_t wn[4];  // the words of the next block
#pragma unroll
                for (int i = 0; i < 4; ++i) wn[i] = lds<uint32_t>(wh + 1024 * i);
                // minus the zero, in 64ths (made as the nibbles are)
                uint32_t zero[4] = {0xBE00BE00u, 0xBE00BE00u, 0xBE00BE00u, 0xBE00BE00u};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b >= left) break;
                    const int group = (4 * half + b) / kPer;
                    if (b % kPer == 0 && a.zeros) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t z =
                                kWholeZeros ? zv[i] : lds<uint8_t>(zd + 8 * i * G::kZeroPitch + group);
                            const uint32_t two =
                                __byte_perm(z, 0, 0x4040 + (kWholeZeros ? 0x0101 * (b / kPer) : 0));
                            zero[i] = fma_bf16x2(two, 0xFF00FF00u, 0);
                        }
                    }
                    // A nibble in the low byte of a BF16 is 2^-133 (or 16 times that) times
                    // its value, linear through the subnormals and the first binade, so one
                    // multiply-add by 2^127 (2^123) gives (q - z) / 64, exact.  The copy's
                    // swizzle keeps the eight columns' words in different banks.
                    uint32_t q[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = wn[i];
                        if (b < 3) wn[i] = lds<uint32_t>((wh ^ (b + 1) << 4) + 1024 * i);
                        const uint32_t v = w >> 8;
                        q[i][0] = fma_bf16x2(w & 0x000F000Fu, 0x7F007F00u, zero[i]);
                        q[i][1] = fma_bf16x2(w & 0x00F000F0u, 0x7D007D00u, zero[i]);
                        q[i][2] = fma_bf16x2(v & 0x000F000Fu, 0x7F007F00u, zero[i]);
                        q[i][3] = fma_bf16x2(v & 0x00F000F0u, 0x7D007D00u, zero[i]);
                    }
                    // q[.][j] holds summed values j and j + 4 of the thread's eight
                    const uint32_t a0[2][4] = {{q[0][0], q[1][0], q[0][1], q[1][1]},
                                               {q[2][0], q[3][0], q[2][1], q[3][1]}};
                    const uint32_t a1[2][4] = {{q[0][2], q[1][2], q[0][3], q[1][3]},
                                               {q[2][2], q[3][2], q[2][3], q[3][3]}};
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 v = xv[b % kAhead][i];
                        const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410);
                        const uint32_t b1 = __byte_perm(v.x, v.z, 0x7632);
                        const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410);
                        const uint32_t b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            if (b % kPer == 0)
                                mma_16816_first(sum[m][i], a0[m], b0, b1);
                            else
                                mma_16816(sum[m][i], a0[m], b0, b1);
                            mma_16816(sum[m][i], a1[m], b2, b3);
                        }
                    }
                    if (b + kAhead < 4) {
                        if (b + kAhead < left) load_x(b + kAhead, 0);
                    } else if (b + kAhead - 4 < after) {
                        load_x(b + kAhead - 4, x_next);
                    }
                    if (b % kPer == kPer - 1) {
                        float s[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t at = sd + 8 * i * G::kScalePitch;
                            s[i] = WHOLE ? __uint_as_float(sv[i][b / kPer])
                                   : a.scale_fp32
                                       ? lds<float>(at + 4 * group)
                                       : __uint_as_float(uint32_t{lds<uint16_t>(at + 2 * group)} << 16);
                        }
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int i = 0; i < NT; ++i)
#pragma unroll
                                for (int j = 0; j < 4; j += 2)
                                    fma_f32x2(acc[m][i][j], acc[m][i][j + 1], s[2 * m + j / 2],
                                              sum[m][i][j], sum[m][i][j + 1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) x[i] += x_next;
            }
            __syncwarp();
            ++it;
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
                    const float v =
                        outside[i] >> (4 * (2 * t + j % 2)) & 1u ? 0.f : 64.f * acc[m][i][j];
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

template <int GROUP, int TILES, bool WHOLE>
__global__ void __launch_bounds__(32 * warps_of(TILES), 1)
    grouped_gemv_int4_kernel(const __grid_constant__ CUtensorMap map, const GemvArgs a,
                             const int share) {
    constexpr int kWarps = warps_of(TILES), kGemvThreads = 32 * kWarps;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + (((smem_u32(raw) + 1023u) & ~1023u) - smem_u32(raw));
    uint8_t *group_data = smem + kWarps * kStages * kWeightBytes;
    uint8_t *sums = group_data + kWarps * kStages * GroupData<GROUP>::kBytes;
    GemvControl &c =
        *reinterpret_cast<GemvControl *>(sums + kWarps * GemvSmem<GROUP, TILES>::kSumBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane < kStages) mbar_init(smem_u32(&c.full[warp][lane]), 1);
    fence_mbar_init();
    pdl_wait();

    const int total = scan_experts<kGemvThreads>(a.offsets, a.num_experts, static_cast<int>(a.rows),
                                                 8 * TILES, c.lo, c.tiles, c.scan);
    __syncthreads();

    const int block = warp / share;
    const unsigned col_blocks = (a.n + kCols - 1) / kCols;
    const int at_once = kWarps / share, items = total * static_cast<int>(col_blocks);
    const int item0 = first_item(block, at_once, items);
    const Gemv<GROUP, TILES, WHOLE> k{a,
                        map,
                        c,
                        lane,
                        lane / 4,
                        lane % 4,
                        share,
                        warp % share,
                        static_cast<int>(gridDim.x) * at_once,
                        items,
                        col_blocks,
                        (a.k + kSpan - 1) / kSpan,
                        a.k / GROUP,
                        1 << (31 - __clz(a.num_experts)),
                        smem_u32(smem) + warp * (kStages * kWeightBytes),
                        smem_u32(group_data) + warp * (kStages * GroupData<GROUP>::kBytes),
                        smem_u32(&c.full[warp][0]),
                        reinterpret_cast<float *>(sums) + block * share * (kCols * 8 * TILES),
                        block};
    Cursor now{item0, k.part, 0, 0, 0, 0};
    k.locate(now);
    Copies ahead{item0, k.part, 0, 0, 0};
    k.locate(ahead);
    for (int s = 0; s < kStages - 1; ++s) k.issue(ahead, s);
    uint32_t it = 0;
    uint64_t limit = a.timeout_ns;
    while (now.item < k.items) {
        if (TILES == 1 || now.rows <= 8)
            k.template item<1>(now, ahead, it, limit);
        else if (TILES <= 2 || now.rows <= 16)
            k.template item<(TILES < 2 ? TILES : 2)>(now, ahead, it, limit);
        else
            k.template item<TILES>(now, ahead, it, limit);
    }
    if (limit == 0)  // copies may still be in flight: wait once more before the memory goes
        for (uint32_t s = 1; s <= kStages && s <= it; ++s)
            (void)mbar_wait_long(k.full + 8 * ((it - s) % kStages), (it - s) / kStages & 1, a.timeout_ns);
    cp_async_wait<0>();
}

template <int GROUP, int TILES, bool WHOLE>
cudaError_t launch(const GemvArgs &a, cudaStream_t s) {
    constexpr int kWarps = warps_of(TILES);
    CUtensorMap map;
    const cuuint64_t row = static_cast<cuuint64_t>(a.k) / 2;
    if (!encode_map(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, 3,
                    {row, static_cast<cuuint64_t>(a.n), static_cast<cuuint64_t>(a.num_experts)},
                    {row, row * a.n}, kSpan / 2, kCols))
        return cudaErrorInvalidValue;
    const int64_t blocks = (a.n + kCols - 1) / kCols *
                           (a.rows / (8 * TILES) + min(int64_t{a.num_experts}, a.rows));
    const int share = warps_of_block(blocks, (a.k + kSpan - 1) / kSpan, kWarps, a.num_sms);
    // work items are counted in 32 bits (a buffer of so many results does not fit)
    if (blocks > INT32_MAX - int64_t{a.num_sms} * kWarps) return cudaErrorInvalidValue;
    return launch_ex(grouped_gemv_int4_kernel<GROUP, TILES, WHOLE>,
                     dim3(static_cast<unsigned>(min(blocks, int64_t{a.num_sms}))),
                     dim3(32 * kWarps), GemvSmem<GROUP, TILES>::kBytes, s, 1, a.programmatic, map, a, share);
}

template <int GROUP>
cudaError_t launch_group(const GemvArgs &a, cudaStream_t s) {
    // Rows of a pass by the average of an expert: 16 above five rows (8 rows 100 against
    // 122 us for 32 a pass), 32 above 24 (one matrix: 24 rows 52 us in passes of 16, 62 in
    // one of 32; 32 rows 80 against 62).
    const bool whole = a.k % kSpan == 0 && reinterpret_cast<uintptr_t>(a.scales) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.zeros) % 8 == 0;
    const int64_t E = a.num_experts;
    if (a.rows > 24 * E) return whole ? launch<GROUP, 4, true>(a, s) : launch<GROUP, 4, false>(a, s);
    if (a.rows > 5 * E) return whole ? launch<GROUP, 2, true>(a, s) : launch<GROUP, 2, false>(a, s);
    return whole ? launch<GROUP, 1, true>(a, s) : launch<GROUP, 1, false>(a, s);
}

template <int GROUP, int TILES>
cudaError_t prepare() {
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const int bytes = GemvSmem<GROUP, TILES>::kBytes;
    const cudaError_t e =
        cudaFuncSetAttribute(grouped_gemv_int4_kernel<GROUP, TILES, false>, attr, bytes);
    return e != cudaSuccess
               ? e
               : cudaFuncSetAttribute(grouped_gemv_int4_kernel<GROUP, TILES, true>, attr, bytes);
}

}  // namespace

template <int GROUP>
static cudaError_t prepare_group() {
    cudaError_t e = prepare<GROUP, 1>();
    if (e == cudaSuccess) e = prepare<GROUP, 2>();
    return e == cudaSuccess ? prepare<GROUP, 4>() : e;
}

cudaError_t prepare_grouped_gemv() {
    cudaError_t e = find_encoder();
    if (e == cudaSuccess) e = prepare_group<32>();
    if (e == cudaSuccess) e = prepare_group<64>();
    return e == cudaSuccess ? prepare_group<128>() : e;
}

cudaError_t launch_grouped_gemv_int4(const GemvArgs &a, cudaStream_t s) {
    switch (a.group) {
        case 32: return launch_group<32>(a, s);
        case 64: return launch_group<64>(a, s);
        default: return launch_group<128>(a, s);
    }
}

}  // namespace mf
