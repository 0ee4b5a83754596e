// Host-side launch interface of the expert-layer kernels (experts_api.cu calls
// them after validation).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mf {

constexpr int kMaxExperts = 1024;

struct PermuteArgs {
    const int32_t *ids;      // [slots] expert ids, or packed words (id << 16 | weight bits)
    int packed;
    int64_t slots;           // T * K
    int top_k;
    int num_experts;
    int32_t *offsets;        // [E + 1]
    int32_t *slot_to_row;    // [slots], -1 for a slot without an expert
    int32_t *row_to_token;   // [slots], -1 behind the last row
    bool programmatic;
};

struct RowSumArgs {
    const void *rows;        // [num_rows, ld] BF16 or FP32
    int rows_fp32;
    int64_t num_rows;
    int64_t ld;
    const int32_t *idx;      // [T, K]
    void *out;               // [T, hidden] BF16 or FP32
    int out_fp32;
    int64_t num_tokens;
    int hidden;
    int top_k;
    bool programmatic;
};

// Which product over the rows of each expert.
enum GroupedKind { kForward = 0, kDgrad = 1, kWgrad = 2 };

struct GroupedArgs {
    int kind;
    const void *x;           // forward, wgrad: BF16 [x_rows, x_ld] rows of K values
    int64_t x_rows;
    int64_t x_ld;
    const int32_t *row_index;  // row of x that product row r reads, or nullptr (row r)
    const void *dy;          // dgrad, wgrad: BF16 [rows, dy_ld] rows of N values
    int64_t dy_ld;
    const void *w;           // forward, dgrad: BF16 [E, N, K]
    int64_t w_ld;            // elements between rows n
    int64_t w_expert;        // elements between experts
    const int32_t *offsets;  // [E + 1]
    int64_t rows;
    int num_experts;
    int n;
    int k;
    void *out;               // forward [rows, N], dgrad [rows, K], wgrad [E, N, K]
    int out_fp32;
    int64_t out_ld;          // forward, dgrad
    int accumulate;          // wgrad: add to what out holds
    int num_sms;
    int num_pairs;           // pairs of SMs that run at once
    unsigned *status;
    uint64_t timeout_ns;
    bool programmatic;
};

struct GemvArgs {
    const void *x;           // BF16 [x_rows, x_ld]
    int64_t x_rows;
    int64_t x_ld;
    const int32_t *row_index;
    const uint8_t *w;        // [E, N, K / 2], low half first
    const void *scales;      // [E, N, K / group] BF16 or FP32
    int scale_fp32;
    const uint8_t *zeros;    // [E, N, K / group] or nullptr (8)
    int group;
    const int32_t *offsets;  // [E + 1], or nullptr: one expert with every row
    int64_t rows;
    int num_experts;
    int n;
    int k;
    void *out;               // [rows, out_ld] BF16 or FP32
    int out_fp32;
    int64_t out_ld;
    int num_sms;
    unsigned *status;
    uint64_t timeout_ns;
    bool programmatic;
};

// Per-device one-time set-up (kernel attributes); `pairs`: clusters of two CTAs
// of the grouped product that the device runs at once.
cudaError_t prepare_expert_kernels(int *pairs);

cudaError_t launch_expert_permutation(const PermuteArgs &a, cudaStream_t s);
cudaError_t launch_permuted_row_sum(const RowSumArgs &a, cudaStream_t s);
cudaError_t launch_grouped_gemm(const GroupedArgs &a, cudaStream_t s);
cudaError_t launch_grouped_gemv_int4(const GemvArgs &a, cudaStream_t s);

}  // namespace mf
