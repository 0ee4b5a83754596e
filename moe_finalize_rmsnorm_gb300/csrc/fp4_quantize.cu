// Rows to 4-bit floating point and back.  For a block of g values (g = 32 or 16) with the
// largest magnitude m of v = factor * x (FP32),
//
//   E8M0 (g = 32)   s = 2^(floor(log2 m) - 2), at least 2^-127
//   E4M3 (g = 16)   s = E4M3(m / 6), at most 448
//   q = E2M1(v / s), nearest, ties to even, at most 6 in magnitude; 0 where s is 0
//
// A block with an infinity or a NaN gets a NaN as its scale and zeros as its values.
//
// Bound by the bytes (16384 rows of 7168, BF16: 47 us for E8M0 and 48 for E4M3, 44 at the
// copy's rate; back 45 and 48), and with E4M3 by the instructions: a thread takes 8 values,
// or 16 that are one block (58 us with 8), so that a warp's loads and stores are one run
// each, and the 2 or 4 threads of a longer block exchange their largest magnitudes.  The
// quotients decide between neighbours as the exact ones do: with an E8M0 scale they are
// exact, and with E4M3 they are rounded as a division's (a reciprocal by one step of
// Newton's iteration, and its product put right by its remainder: Markstein's correction of
// a quotient).  A quotient next to a border between two codes differs from it by more than
// half a step of FP32, as border times scale has at most 7 bits, and a product with the
// reciprocal alone would miss some of the ties themselves.
#include "fp4.cuh"
#include "rows.cuh"

namespace mf {
namespace {

constexpr int kThreads = 128;
constexpr int kChunks = 4;  // for each thread

// Values of a chunk: 16 bytes, or the 32 of an E4M3 block in BF16.
template <int FORMAT, bool X_FP32>
constexpr int kValues = FORMAT == kNv && !X_FP32 ? 16 : 8;

// Row and column of chunk `at` (0 .. 511) of the block's; `values` to a chunk.
struct Place {
    int64_t row;
    int col;
};

__device__ __forceinline__ Place place_of(const Fp4RowsArgs &a, int chunks, int64_t first_row,
                                          int first, int at, int values) {
    const uint32_t n = first + at;
    // below 2^10 with up to 512 chunks a row: the product's error stays below one row
    const uint32_t over = chunks <= 512 ? __umulhi(n, a.magic) : n >= static_cast<uint32_t>(chunks);
    return {first_row + over, static_cast<int>(n - over * chunks) * values};
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return r;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return r;
}

// 1 / s, rounded, of the values of E4M3: the hardware's estimate and one step of Newton's
// iteration.
__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    return fmaf(fmaf(-s, r, 1.f), r, r);
}

// 32 bytes at once, where they lie on a multiple of 32 (`wide`).
__device__ __forceinline__ void load_32(const uint8_t *p, bool read, bool wide, uint4 (&v)[2]) {
    if (wide) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %9, 0;\n\t"
            "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
            "mov.u32 %4, 0;\n\tmov.u32 %5, 0;\n\tmov.u32 %6, 0;\n\tmov.u32 %7, 0;\n\t"
            "@p ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t}"
            : "=&r"(v[0].x), "=&r"(v[0].y), "=&r"(v[0].z), "=&r"(v[0].w), "=&r"(v[1].x),
              "=&r"(v[1].y), "=&r"(v[1].z), "=&r"(v[1].w)
            : "l"(p), "r"(uint32_t{read}));
    } else {
        v[0] = ld_nc_na_16_if(p, read);
        v[1] = ld_nc_na_16_if(p + 16, read);
    }
}

__device__ __forceinline__ uint32_t largest_bf16(const uint4 &w) {
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
}

template <int FORMAT, bool X_FP32, bool FACTOR>
__global__ void __launch_bounds__(kThreads) quantize_fp4_kernel(Fp4RowsArgs a) {
    constexpr int N = kValues<FORMAT, X_FP32>;
    constexpr int kBlock = FORMAT == kMx ? 32 : 16;
    constexpr bool kTwo = X_FP32 || N == 16;  // 16-byte pieces of a chunk: two
    pdl_wait();
    const int chunks = a.k / N;
    const int64_t begin = int64_t{blockIdx.x} * (kThreads * kChunks);
    const int64_t first_row = begin / chunks;
    const int first = static_cast<int>(begin - first_row * chunks);
    uint4 x[kChunks][kTwo ? 2 : 1];
    Place p[kChunks];
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        p[u] = place_of(a, chunks, first_row, first, u * kThreads + threadIdx.x, N);
        const uint8_t *from = static_cast<const uint8_t *>(a.x) +
                              (p[u].row * a.x_ld + p[u].col) * (X_FP32 ? 4 : 2);
        const bool read = p[u].row < a.rows;
        if constexpr (kTwo)
            load_32(from, read, a.wide, x[u]);
        else
            x[u][0] = ld_nc_na_16_if(from, read);
    }
    const float factor = FACTOR ? __ldg(a.factor) : 1.f;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint4 &w = x[u][i / (X_FP32 ? 4 : 8)];
            const int at = X_FP32 ? i % 4 : i % 8 / 2;
            const uint32_t bits = at == 0 ? w.x : at == 1 ? w.y : at == 2 ? w.z : w.w;
            v[i] = X_FP32 ? __uint_as_float(bits) : i % 2 ? bf16_hi(bits) : bf16_lo(bits);
        }
        // Magnitudes as integers: their order is the values', with the infinity and NaNs on top;
        // and the largest product's is the product of the largest, as rounding keeps the order.
        uint32_t top = 0;
        if (X_FP32) {
#pragma unroll
            for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        } else {
            top = largest_bf16(x[u][0]);
            if (N == 16) top = max(top, largest_bf16(x[u][kTwo ? 1 : 0]));
        }
#pragma unroll
        for (int across = 1; across < kBlock / N; across *= 2)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, across));
        if (FACTOR) top = __float_as_uint(__uint_as_float(top) * factor) & 0x7fffffffu;
        uint32_t byte;
        float2 r2, s2 = make_float2(0.f, 0.f);
        if (FORMAT == kMx) {
            const int e = static_cast<int>(top >> 23);
            byte = max(e - 2, 0);
            const float r = __uint_as_float((254u - byte) << 23);
            r2 = make_float2(r, r);
        } else {
            // top / 6, rounded as a division's: Markstein's correction
            const float m = __uint_as_float(top);
            constexpr float kSixth = 1.f / 6.f;
            const float c = m * kSixth;
            const float want = fmaf(fmaf(-c, 6.f, m), kSixth, c);
            byte = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
            const float s = scale_of<kNv>(byte);
            const float r = byte == 0 ? 0.f : reciprocal(s);
            r2 = make_float2(r, r);
            s2 = make_float2(s, s);
        }
        const bool bad = top >= 0x7f800000u;
        if (bad) byte = FORMAT == kMx ? 0xffu : 0x7fu;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float2 y = make_float2(v[i], v[i + 1]);
            if (FACTOR) y = mul2(y, make_float2(factor, factor));
            float2 q = mul2(y, r2);
            if (FORMAT == kNv)  // (a zero keeps its sign in this form of the remainder)
                q = fma2(fma2(q, s2, make_float2(-y.x, -y.y)), make_float2(-r2.x, -r2.y), q);
            v[i] = q.x;
            v[i + 1] = q.y;
        }
        if (p[u].row >= a.rows) continue;
        uint8_t *to = a.q + p[u].row * a.q_ld + p[u].col / 2;
        if constexpr (N == 16) {
            const float(&low)[8] = reinterpret_cast<const float(&)[8]>(v[0]);
            const float(&high)[8] = reinterpret_cast<const float(&)[8]>(v[8]);
            *reinterpret_cast<uint2 *>(to) =
                bad ? make_uint2(0, 0) : make_uint2(to_e2m1(low), to_e2m1(high));
        } else {
            *reinterpret_cast<uint32_t *>(to) = bad ? 0u : to_e2m1(v);
        }
        if (p[u].col % kBlock == 0)
            a.scales[p[u].row * a.s_ld + p[u].col / kBlock] = static_cast<uint8_t>(byte);
    }
}

template <int FORMAT, bool OUT_FP32>
__global__ void __launch_bounds__(kThreads) dequantize_fp4_kernel(Fp4RowsArgs a) {
    pdl_wait();
    const int chunks = a.k / 8;
    const int64_t begin = int64_t{blockIdx.x} * (kThreads * kChunks);
    const int64_t first_row = begin / chunks;
    const int first = static_cast<int>(begin - first_row * chunks);
    constexpr int kBlock = FORMAT == kMx ? 32 : 16;
    Place p[kChunks];
    uint32_t q[kChunks], s[kChunks];
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        p[u] = place_of(a, chunks, first_row, first, u * kThreads + threadIdx.x, 8);
        q[u] = s[u] = 0;
        if (p[u].row < a.rows) {
            q[u] = __ldg(reinterpret_cast<const uint32_t *>(a.q + p[u].row * a.q_ld + p[u].col / 2));
            s[u] = __ldg(a.scales + p[u].row * a.s_ld + p[u].col / kBlock);
        }
    }
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        if (p[u].row >= a.rows) continue;
        uint32_t h[4];
        from_e2m1(q[u], h);
        const float scale = scale_of<FORMAT>(s[u]);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            v[2 * i] = f.x * scale;
            v[2 * i + 1] = f.y * scale;
        }
        if (OUT_FP32 && a.wide)  // whole 32-byte sectors
            asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             static_cast<float *>(a.out) + p[u].row * a.out_ld + p[u].col),
                         "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]),
                         "f"(v[6]), "f"(v[7])
                         : "memory");
        else
            store8<OUT_FP32>(a.out, p[u].row * a.out_ld + p[u].col, v);
    }
}

bool on_32_bytes(const void *p, int64_t stride_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && stride_bytes % 32 == 0;
}

template <typename K>
cudaError_t go(K kernel, int values, const Fp4RowsArgs &a, cudaStream_t s) {
    const int64_t chunks = a.k / values, per_block = kThreads * kChunks;
    Fp4RowsArgs b = a;
    b.wide = a.x ? on_32_bytes(a.x, a.x_ld * (a.x_fp32 ? 4 : 2))
                 : on_32_bytes(a.out, a.out_ld * (a.out_fp32 ? 4 : 2));
    b.magic = static_cast<uint32_t>((0x100000000ull + chunks - 1) / chunks);
    return launch_ex(kernel, dim3(static_cast<unsigned>((a.rows * chunks + per_block - 1) / per_block)),
                     dim3(kThreads), 0, s, 1, a.programmatic, b);
}

template <int FORMAT>
cudaError_t quantize(const Fp4RowsArgs &a, cudaStream_t s) {
    if (a.x_fp32)
        return a.factor ? go(quantize_fp4_kernel<FORMAT, true, true>, 8, a, s)
                        : go(quantize_fp4_kernel<FORMAT, true, false>, 8, a, s);
    constexpr int N = kValues<FORMAT, false>;
    return a.factor ? go(quantize_fp4_kernel<FORMAT, false, true>, N, a, s)
                    : go(quantize_fp4_kernel<FORMAT, false, false>, N, a, s);
}

}  // namespace

cudaError_t launch_quantize_fp4(const Fp4RowsArgs &a, cudaStream_t s) {
    return a.format == kMx ? quantize<kMx>(a, s) : quantize<kNv>(a, s);
}

cudaError_t launch_dequantize_fp4(const Fp4RowsArgs &a, cudaStream_t s) {
    if (a.format == kMx)
        return a.out_fp32 ? go(dequantize_fp4_kernel<kMx, true>, 8, a, s)
                          : go(dequantize_fp4_kernel<kMx, false>, 8, a, s);
    return a.out_fp32 ? go(dequantize_fp4_kernel<kNv, true>, 8, a, s)
                      : go(dequantize_fp4_kernel<kNv, false>, 8, a, s);
}

}  // namespace mf
