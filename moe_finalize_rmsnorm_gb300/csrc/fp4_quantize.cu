// Rows to 4-bit floating point and back.  For a block of g values (g = 32 or 16) with the
// largest magnitude m of v = factor * x (FP32),
//
//   E8M0 (g = 32)   s = 2^(floor(log2 m) - 2), at least 2^-127
//   E4M3 (g = 16)   s = E4M3(m / 6), at most 448
//   q = E2M1(v / s), nearest, ties to even, at most 6 in magnitude; 0 where s is 0
//
// A block with an infinity or a NaN gets a NaN as its scale and zeros as its values.
//
// Bound by the bytes: a thread takes 8 values, so that a warp's loads and stores are one
// run each, and the 2 or 4 threads of a block exchange their largest magnitudes.  The
// quotients decide between neighbours as the exact ones do: with an E8M0 scale they are
// exact, and with E4M3 they are rounded as a division's (a reciprocal's product, put right
// by its remainder): a quotient next to a border between two codes differs from it by
// more than half a step of FP32, as border times scale has at most 7 bits, and a product
// with the reciprocal alone would miss some of the ties themselves.
#include "fp4.cuh"
#include "rows.cuh"

namespace mf {
namespace {

constexpr int kThreads = 128;
constexpr int kChunks = 4;  // of 8 values, for each thread

// Row and column of chunk `at` (0 .. 511) of the block's.
struct Place {
    int64_t row;
    int col;
};

__device__ __forceinline__ Place place_of(const Fp4RowsArgs &a, int chunks, int64_t first_row,
                                          int first, int at) {
    const uint32_t n = first + at;
    // below 2^10 with up to 512 chunks a row: the product's error stays below one row
    const uint32_t over = chunks <= 512 ? __umulhi(n, a.magic) : n >= static_cast<uint32_t>(chunks);
    return {first_row + over, static_cast<int>(n - over * chunks) * 8};
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

template <int FORMAT, bool X_FP32, bool FACTOR>
__global__ void __launch_bounds__(kThreads) quantize_fp4_kernel(Fp4RowsArgs a) {
    pdl_wait();
    const int chunks = a.k / 8;
    const int64_t begin = int64_t{blockIdx.x} * (kThreads * kChunks);
    const int64_t first_row = begin / chunks;
    const int first = static_cast<int>(begin - first_row * chunks);
    Chunk8<X_FP32> x[kChunks];
    Place p[kChunks];
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        p[u] = place_of(a, chunks, first_row, first, u * kThreads + threadIdx.x);
        x[u].load(a.x, p[u].row * a.x_ld + p[u].col, p[u].row < a.rows);
    }
    const float factor = FACTOR ? __ldg(a.factor) : 1.f;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        float v[8];
        x[u].get(v);
        // magnitudes as integers: their order is the values', with the infinity and NaNs on top
        uint32_t top = 0;
        if (X_FP32 || FACTOR) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (FACTOR) v[i] *= factor;
                top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
            }
        } else {
            const uint4 &w = x[u].v[0];
            const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                        __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
            top = max(m << 16, m & 0xffff0000u);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if (FORMAT == kMx) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        uint32_t byte;
        float2 r2, s2 = make_float2(0.f, 0.f);
        if (FORMAT == kMx) {
            const int e = static_cast<int>(top >> 23);
            byte = max(e - 2, 0);
            const float r = __uint_as_float((254u - byte) << 23);
            r2 = make_float2(r, r);
        } else {
            // top / 6, rounded as a division's
            const float m = __uint_as_float(top);
            constexpr float kSixth = 1.f / 6.f;
            const float c = m * kSixth;
            const float want = fmaf(fmaf(-c, 6.f, m), kSixth, c);
            byte = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
            const float s = scale_of<kNv>(byte);
            const float r = byte == 0 ? 0.f : __frcp_rn(s);
            r2 = make_float2(r, r);
            s2 = make_float2(s, s);
        }
        if (top >= 0x7f800000u) {
            byte = FORMAT == kMx ? 0xffu : 0x7fu;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
            r2 = s2 = make_float2(0.f, 0.f);  // these may be NaN, too
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 y = make_float2(v[i], v[i + 1]);
            float2 q = mul2(y, r2);
            if (FORMAT == kNv)  // (a zero keeps its sign in this form of the remainder)
                q = fma2(fma2(q, s2, make_float2(-y.x, -y.y)), make_float2(-r2.x, -r2.y), q);
            v[i] = q.x;
            v[i + 1] = q.y;
        }
        if (p[u].row >= a.rows) continue;
        *reinterpret_cast<uint32_t *>(a.q + p[u].row * a.q_ld + p[u].col / 2) = to_e2m1(v);
        constexpr int kBlock = FORMAT == kMx ? 32 : 16;
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
        p[u] = place_of(a, chunks, first_row, first, u * kThreads + threadIdx.x);
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
        store8<OUT_FP32>(a.out, p[u].row * a.out_ld + p[u].col, v);
    }
}

template <typename K>
cudaError_t go(K kernel, const Fp4RowsArgs &a, cudaStream_t s) {
    const int64_t chunks = a.k / 8, per_block = kThreads * kChunks;
    Fp4RowsArgs b = a;
    b.magic = static_cast<uint32_t>((0x100000000ull + chunks - 1) / chunks);
    return launch_ex(kernel, dim3(static_cast<unsigned>((a.rows * chunks + per_block - 1) / per_block)),
                     dim3(kThreads), 0, s, 1, a.programmatic, b);
}

template <int FORMAT>
cudaError_t quantize(const Fp4RowsArgs &a, cudaStream_t s) {
    if (a.x_fp32)
        return a.factor ? go(quantize_fp4_kernel<FORMAT, true, true>, a, s)
                        : go(quantize_fp4_kernel<FORMAT, true, false>, a, s);
    return a.factor ? go(quantize_fp4_kernel<FORMAT, false, true>, a, s)
                    : go(quantize_fp4_kernel<FORMAT, false, false>, a, s);
}

}  // namespace

cudaError_t launch_quantize_fp4(const Fp4RowsArgs &a, cudaStream_t s) {
    return a.format == kMx ? quantize<kMx>(a, s) : quantize<kNv>(a, s);
}

cudaError_t launch_dequantize_fp4(const Fp4RowsArgs &a, cudaStream_t s) {
    if (a.format == kMx)
        return a.out_fp32 ? go(dequantize_fp4_kernel<kMx, true>, a, s)
                          : go(dequantize_fp4_kernel<kMx, false>, a, s);
    return a.out_fp32 ? go(dequantize_fp4_kernel<kNv, true>, a, s)
                      : go(dequantize_fp4_kernel<kNv, false>, a, s);
}

}  // namespace mf
