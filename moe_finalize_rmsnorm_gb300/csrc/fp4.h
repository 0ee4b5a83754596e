// Host-side launch interface of the 4-bit floating point kernels (fp4_api.cu calls
// them after validation).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mf {

// Values are E2M1, two to a byte (the even column in the low half).  kMx: a block of 32
// columns has a power of two as its scale (E8M0); kNv: a block of 16 a scale in E4M3.
enum Fp4Format { kMx = 0, kNv = 1 };

struct Fp4RowsArgs {
    const void *x;         // quantize: BF16 or FP32 [rows, x_ld]
    int64_t x_ld;
    int x_fp32;
    const float *factor;   // x is multiplied by it first, or nullptr
    uint8_t *q;            // [rows, q_ld] bytes
    int64_t q_ld;
    uint8_t *scales;       // [rows, s_ld] bytes
    int64_t s_ld;
    void *out;             // dequantize: BF16 or FP32 [rows, out_ld]
    int64_t out_ld;
    int out_fp32;
    int format;
    int64_t rows;
    int k;
    uint32_t magic;        // 2^32 / (chunks of a row), for few chunks (set by the launch)
    bool wide;             // x, or the output, in accesses of 32 bytes (set by the launch)
    bool programmatic;
};

struct Fp4GemmArgs {
    const uint8_t *x;          // [x_rows, x_ld] bytes
    int64_t x_rows;
    int64_t x_ld;
    const uint8_t *x_scales;   // [x_rows, xs_ld] bytes
    int64_t xs_ld;
    const int32_t *row_index;  // row of x that product row r reads, or nullptr (row r)
    const uint8_t *w;          // [E, n] rows of w_ld bytes, experts w_expert bytes apart
    int64_t w_ld;
    int64_t w_expert;
    const uint8_t *w_scales;   // [E, n] rows of ws_ld bytes, experts ws_expert bytes apart
    int64_t ws_ld;
    int64_t ws_expert;
    const float *factor;       // [E] of the results, or nullptr
    const int32_t *offsets;    // [E + 1], or nullptr: one expert with every row
    int format;
    int64_t rows;
    int num_experts;
    int n;
    int k;
    void *out;                 // [rows, out_ld] BF16 or FP32
    int out_fp32;
    int64_t out_ld;
    int num_sms;
    int num_pairs;             // pairs of SMs that run at once
    unsigned *status;
    uint64_t timeout_ns;
    bool programmatic;
};

cudaError_t launch_quantize_fp4(const Fp4RowsArgs &a, cudaStream_t s);
cudaError_t launch_dequantize_fp4(const Fp4RowsArgs &a, cudaStream_t s);

cudaError_t prepare_fp4_gemm(int *pairs);
cudaError_t prepare_fp4_rows();
cudaError_t launch_fp4_gemm(const Fp4GemmArgs &a, cudaStream_t s);
// The same for few rows (launch_fp4_gemm chooses it).
cudaError_t launch_fp4_rows(const Fp4GemmArgs &a, cudaStream_t s);

}  // namespace mf
