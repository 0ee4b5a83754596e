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
    bool wide_clusters;      // the device runs clusters of 16
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

// Whether a forward product takes the kernel for few rows: up to 64 rows, or two an
// expert (the experts' own are known on the device only; 256 at most, for a router that
// sends them all to one).  At 2048 x 4096, few-rows against tensor-core kernel: 2 rows
// 9 against 21 us, 8 rows 23.3 against 27.0, 64 rows of 64 experts 108 against 116, 128
// rows of 64 experts 134 against 141, 64 rows of 8 experts 27.7 against 27.8, 256 rows of
// 8 experts 53 against 28.
inline bool few_rows(int64_t rows, int num_experts) {
    return rows <= 64 || (rows <= 256 && rows <= 2 * int64_t{num_experts});
}

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
    int sum_from, sum_to;    // wgrad: experts with so many rows (set by the launch)
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

// Per-device one-time set-up of each family (kernel attributes).  `wide_clusters`:
// whether the device runs clusters of 16; `pairs`: clusters of two CTAs of the grouped
// product that it runs at once.
cudaError_t prepare_permute_kernels(bool *wide_clusters);
cudaError_t prepare_grouped_gemm(int *pairs);
cudaError_t prepare_grouped_rows();
cudaError_t prepare_grouped_gemv();

cudaError_t launch_expert_permutation(const PermuteArgs &a, cudaStream_t s);
cudaError_t launch_permuted_row_sum(const RowSumArgs &a, cudaStream_t s);
cudaError_t launch_grouped_gemm(const GroupedArgs &a, cudaStream_t s);
// The same for few rows (forward; launch_grouped_gemm chooses it).
cudaError_t launch_grouped_rows(const GroupedArgs &a, cudaStream_t s);
cudaError_t launch_grouped_gemv_int4(const GemvArgs &a, cudaStream_t s);

}  // namespace mf
