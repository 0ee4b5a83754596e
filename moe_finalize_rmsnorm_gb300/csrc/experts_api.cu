// C ABI of the expert-layer operations: argument validation and launches.
// Declarations and the contract are in include/moe_finalize.h.
#include <cuda_runtime.h>

#include <mutex>

#include "device_info.h"
#include "experts.h"
#include "moe_finalize.h"

namespace {

using mf::aligned;

constexpr int64_t kMaxRows = 0x7fffffffLL - 1024;  // row numbers and tile ends stay in int32
constexpr int32_t kMaxWidth = 1 << 20;             // columns of a matrix

mf_status from_launch(cudaError_t e) { return e == cudaSuccess ? MF_OK : MF_ERR_CUDA; }

bool value_dtype(mf_dtype d) { return d == MF_DTYPE_BF16 || d == MF_DTYPE_FP32; }

// Row strides of the 16-byte kernels: at least the row, a multiple of 8 elements.
bool row_stride_ok(int64_t stride, int64_t width) {
    return stride >= width && stride % 8 == 0 && stride < (int64_t{1} << 36);
}

// Experts' matrices of rows * width elements: unit stride inside a row, no
// expert inside another.
bool weight_strides_ok(int64_t row_stride, int64_t expert_stride, int32_t num_experts, int32_t n,
                       int32_t k) {
    if (!row_stride_ok(row_stride, k) || !row_stride_ok(expert_stride, 0)) return false;
    return num_experts == 1 || expert_stride >= (n - 1) * row_stride + k;
}

// Whether two buffers share a byte.
bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + static_cast<uintptr_t>(b_bytes) && q < p + static_cast<uintptr_t>(a_bytes);
}

mf_status check_experts(int32_t num_experts, int32_t n, int32_t k) {
    if (num_experts < 1 || num_experts > mf::kMaxExperts) return MF_ERR_UNSUPPORTED;
    if (n < 8 || n > kMaxWidth || n % 8 != 0 || k < 8 || k > kMaxWidth || k % 8 != 0)
        return MF_ERR_UNSUPPORTED;
    return MF_OK;
}

// Each family's kernels are set up on its first call on a device, so that a call of
// another operation pays nothing for them.
enum Family { kPermutation = 1, kProducts = 2, kInt4 = 4 };

struct ExpertDevice {
    unsigned ready = 0;          // families
    bool wide_clusters = false;  // clusters of 16 CTAs run
    int num_pairs = 0;           // resident pairs of SMs of the grouped products
};

constexpr int kMaxDevices = 64;
std::mutex g_expert_mutex;
ExpertDevice g_expert_devices[kMaxDevices];

mf_status expert_device(Family family, const mf::DeviceInfo **info, const ExpertDevice **out) {
    const mf_status st = mf::device_info(info);
    if (st != MF_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MF_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_expert_mutex);
    ExpertDevice &d = g_expert_devices[dev];
    if (!(d.ready & family)) {
        cudaError_t e = cudaSuccess;
        if (family == kPermutation) {
            e = mf::prepare_permute_kernels(&d.wide_clusters);
        } else if (family == kProducts) {
            e = mf::prepare_grouped_gemm(&d.num_pairs);
            if (e == cudaSuccess) e = mf::prepare_grouped_rows();
        } else {
            e = mf::prepare_grouped_gemv();
        }
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return MF_ERR_CUDA;
        }
        d.ready |= family;
    }
    *out = &d;
    return MF_OK;
}

// The facts every grouped launch needs.
mf_status fill(mf::GroupedArgs &a) {
    const mf::DeviceInfo *d = nullptr;
    const ExpertDevice *x = nullptr;
    mf_status st = expert_device(kProducts, &d, &x);
    if (st != MF_OK) return st;
    a.num_sms = d->num_sms;
    a.num_pairs = x->num_pairs;
    a.status = d->status;
    a.timeout_ns = mf::kWaitLimitNs;
    a.programmatic = mf::programmatic_launch();
    return MF_OK;
}

}  // namespace

extern "C" {

mf_status moe_expert_permutation(const int32_t *expert_ids, int packed, int64_t num_tokens,
                                 int32_t top_k, int32_t num_experts, int32_t *expert_offsets,
                                 int32_t *expanded_idx_to_permuted_idx,
                                 int32_t *permuted_row_to_token, mf_stream_t stream) {
    if (num_experts < 1 || num_experts > mf::kMaxExperts || top_k < 1 || top_k > 32)
        return MF_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_tokens > kMaxRows / top_k) return MF_ERR_SHAPE;
    if (!expert_offsets ||
        (num_tokens > 0 && (!expert_ids || !expanded_idx_to_permuted_idx || !permuted_row_to_token)))
        return MF_ERR_NULL;
    if (!aligned(expert_ids, 4) || !aligned(expert_offsets, 4) ||
        !aligned(expanded_idx_to_permuted_idx, 4) || !aligned(permuted_row_to_token, 4))
        return MF_ERR_ALIGN;
    // A map written over ids that are still to be read would not count them as it places
    // them: rows outside the buffers.
    const void *buffers[4] = {expert_ids, expanded_idx_to_permuted_idx, permuted_row_to_token,
                              expert_offsets};
    const int64_t slots = 4 * num_tokens * top_k, bytes[4] = {slots, slots, slots,
                                                              4 * (int64_t{num_experts} + 1)};
    for (int i = 0; num_tokens > 0 && i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(buffers[i], bytes[i], buffers[j], bytes[j])) return MF_ERR_ALIGN;
    const mf::DeviceInfo *d = nullptr;
    const ExpertDevice *x = nullptr;
    mf_status st = expert_device(kPermutation, &d, &x);
    if (st != MF_OK) return st;
    mf::PermuteArgs a = {};
    a.ids = expert_ids;
    a.packed = packed ? 1 : 0;
    a.slots = num_tokens * top_k;
    a.top_k = top_k;
    a.num_experts = num_experts;
    a.offsets = expert_offsets;
    a.slot_to_row = expanded_idx_to_permuted_idx;
    a.row_to_token = permuted_row_to_token;
    a.wide_clusters = x->wide_clusters;
    a.programmatic = mf::programmatic_launch();
    return from_launch(
        mf::launch_expert_permutation(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_permuted_row_sum(const void *permuted, mf_dtype permuted_dtype, int64_t rows,
                               int64_t row_stride, const int32_t *expanded_idx_to_permuted_idx,
                               void *output, mf_dtype output_dtype, int64_t num_tokens,
                               int32_t hidden, int32_t top_k, mf_stream_t stream) {
    if (hidden < 8 || hidden > kMaxWidth || hidden % 8 != 0 || top_k < 1 || top_k > 32)
        return MF_ERR_UNSUPPORTED;
    if (rows < 0 || num_tokens < 0 || num_tokens > kMaxRows / top_k ||
        !row_stride_ok(row_stride, hidden))
        return MF_ERR_SHAPE;
    if (!value_dtype(permuted_dtype) || !value_dtype(output_dtype)) return MF_ERR_DTYPE;
    if (num_tokens == 0) return MF_OK;
    if (!expanded_idx_to_permuted_idx || !output || (rows > 0 && !permuted)) return MF_ERR_NULL;
    if (!aligned(permuted, 16) || !aligned(expanded_idx_to_permuted_idx, 4) || !aligned(output, 16))
        return MF_ERR_ALIGN;
    if ((num_tokens * (hidden / 8) + 127) / 128 > 0x7fffffffLL) return MF_ERR_SHAPE;
    const mf::DeviceInfo *d = nullptr;
    mf_status st = mf::device_info(&d);
    if (st != MF_OK) return st;
    mf::RowSumArgs a = {};
    a.rows = permuted;
    a.rows_fp32 = permuted_dtype == MF_DTYPE_FP32;
    a.num_rows = rows;
    a.ld = row_stride;
    a.idx = expanded_idx_to_permuted_idx;
    a.out = output;
    a.out_fp32 = output_dtype == MF_DTYPE_FP32;
    a.num_tokens = num_tokens;
    a.hidden = hidden;
    a.top_k = top_k;
    a.programmatic = mf::programmatic_launch();
    return from_launch(mf::launch_permuted_row_sum(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_grouped_gemm(const void *x, int64_t x_rows, int64_t x_stride,
                           const int32_t *row_index, const void *weight, int64_t weight_row_stride,
                           int64_t weight_expert_stride, const int32_t *expert_offsets,
                           void *output, mf_dtype output_dtype, int64_t output_stride, int64_t rows,
                           int32_t num_experts, int32_t n, int32_t k, mf_stream_t stream) {
    mf_status st = check_experts(num_experts, n, k);
    if (st != MF_OK) return st;
    if (rows < 0 || rows > kMaxRows || x_rows < 0 || x_rows > kMaxRows ||
        x_rows < (row_index ? (rows > 0) : rows))
        return MF_ERR_SHAPE;
    if (!row_stride_ok(x_stride, k) || !row_stride_ok(output_stride, n) ||
        !weight_strides_ok(weight_row_stride, weight_expert_stride, num_experts, n, k))
        return MF_ERR_SHAPE;
    if (!value_dtype(output_dtype)) return MF_ERR_DTYPE;
    if (rows == 0) return MF_OK;
    if (!x || !weight || !expert_offsets || !output) return MF_ERR_NULL;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(output, 16) ||
        !aligned(expert_offsets, 4) || !aligned(row_index, 4))
        return MF_ERR_ALIGN;
    mf::GroupedArgs a = {};
    st = fill(a);
    if (st != MF_OK) return st;
    a.kind = mf::kForward;
    a.x = x;
    a.x_rows = x_rows;
    a.x_ld = x_stride;
    a.row_index = row_index;
    a.w = weight;
    a.w_ld = weight_row_stride;
    a.w_expert = num_experts > 1 ? weight_expert_stride : weight_row_stride;  // not used by one
    a.offsets = expert_offsets;
    a.rows = rows;
    a.num_experts = num_experts;
    a.n = n;
    a.k = k;
    a.out = output;
    a.out_fp32 = output_dtype == MF_DTYPE_FP32;
    a.out_ld = output_stride;
    return from_launch(mf::launch_grouped_gemm(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_grouped_gemm_dgrad(const void *grad_output, int64_t grad_output_stride,
                                 const void *weight, int64_t weight_row_stride,
                                 int64_t weight_expert_stride, const int32_t *expert_offsets,
                                 void *grad_input, mf_dtype grad_input_dtype,
                                 int64_t grad_input_stride, int64_t rows, int32_t num_experts,
                                 int32_t n, int32_t k, mf_stream_t stream) {
    mf_status st = check_experts(num_experts, n, k);
    if (st != MF_OK) return st;
    if (rows < 0 || rows > kMaxRows) return MF_ERR_SHAPE;
    if (!row_stride_ok(grad_output_stride, n) || !row_stride_ok(grad_input_stride, k) ||
        !weight_strides_ok(weight_row_stride, weight_expert_stride, num_experts, n, k))
        return MF_ERR_SHAPE;
    if (!value_dtype(grad_input_dtype)) return MF_ERR_DTYPE;
    if (rows == 0) return MF_OK;
    if (!grad_output || !weight || !expert_offsets || !grad_input) return MF_ERR_NULL;
    if (!aligned(grad_output, 16) || !aligned(weight, 16) || !aligned(grad_input, 16) ||
        !aligned(expert_offsets, 4))
        return MF_ERR_ALIGN;
    mf::GroupedArgs a = {};
    st = fill(a);
    if (st != MF_OK) return st;
    a.kind = mf::kDgrad;
    a.dy = grad_output;
    a.dy_ld = grad_output_stride;
    a.w = weight;
    a.w_ld = weight_row_stride;
    a.w_expert = num_experts > 1 ? weight_expert_stride : weight_row_stride;  // not used by one
    a.offsets = expert_offsets;
    a.rows = rows;
    a.num_experts = num_experts;
    a.n = n;
    a.k = k;
    a.out = grad_input;
    a.out_fp32 = grad_input_dtype == MF_DTYPE_FP32;
    a.out_ld = grad_input_stride;
    return from_launch(mf::launch_grouped_gemm(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_grouped_gemm_wgrad(const void *grad_output, int64_t grad_output_stride, const void *x,
                                 int64_t x_rows, int64_t x_stride, const int32_t *row_index,
                                 const int32_t *expert_offsets, void *grad_weight,
                                 mf_dtype grad_weight_dtype, int accumulate, int64_t rows,
                                 int32_t num_experts, int32_t n, int32_t k, mf_stream_t stream) {
    mf_status st = check_experts(num_experts, n, k);
    if (st != MF_OK) return st;
    if (rows < 0 || rows > kMaxRows || x_rows < 0 || x_rows > kMaxRows ||
        x_rows < (row_index ? (rows > 0) : rows))
        return MF_ERR_SHAPE;
    if (!row_stride_ok(grad_output_stride, n) || !row_stride_ok(x_stride, k)) return MF_ERR_SHAPE;
    if (!value_dtype(grad_weight_dtype)) return MF_ERR_DTYPE;
    if (!grad_weight || (rows > 0 && (!grad_output || !x || !expert_offsets))) return MF_ERR_NULL;
    if (!aligned(grad_output, 16) || !aligned(x, 16) || !aligned(grad_weight, 16) ||
        !aligned(expert_offsets, 4) || !aligned(row_index, 4))
        return MF_ERR_ALIGN;
    if (rows == 0 && accumulate) return MF_OK;
    mf::GroupedArgs a = {};
    st = fill(a);
    if (st != MF_OK) return st;
    if (rows == 0)  // no row anywhere: every expert's gradient is zero
        return from_launch(cudaMemsetAsync(
            grad_weight, 0,
            size_t{grad_weight_dtype == MF_DTYPE_FP32 ? 4u : 2u} * num_experts * n * k,
            reinterpret_cast<cudaStream_t>(stream)));
    a.kind = mf::kWgrad;
    a.dy = grad_output;
    a.dy_ld = grad_output_stride;
    a.x = x;
    a.x_rows = x_rows;
    a.x_ld = x_stride;
    a.row_index = row_index;
    a.offsets = expert_offsets;
    a.rows = rows;
    a.num_experts = num_experts;
    a.n = n;
    a.k = k;
    a.out = grad_weight;
    a.out_fp32 = grad_weight_dtype == MF_DTYPE_FP32;
    a.accumulate = accumulate ? 1 : 0;
    return from_launch(mf::launch_grouped_gemm(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_grouped_gemv_int4(const void *x, int64_t x_rows, int64_t x_stride,
                                const int32_t *row_index, const uint8_t *weight,
                                const void *scales, mf_dtype scales_dtype, const uint8_t *zeros,
                                int32_t group_size, const int32_t *expert_offsets, void *output,
                                mf_dtype output_dtype, int64_t output_stride, int64_t rows,
                                int32_t num_experts, int32_t n, int32_t k, mf_stream_t stream) {
    if (num_experts < 1 || num_experts > mf::kMaxExperts || n < 1 || n > kMaxWidth || k < 32 ||
        k > kMaxWidth)
        return MF_ERR_UNSUPPORTED;
    if (group_size != 32 && group_size != 64 && group_size != 128) return MF_ERR_UNSUPPORTED;
    if (k % group_size != 0) return MF_ERR_UNSUPPORTED;
    if (rows < 0 || rows > kMaxRows || x_rows < 0 || x_rows > kMaxRows ||
        x_rows < (row_index ? (rows > 0) : rows))
        return MF_ERR_SHAPE;
    if (!row_stride_ok(x_stride, k) || output_stride < n || output_stride >= (int64_t{1} << 36))
        return MF_ERR_SHAPE;
    if (!value_dtype(scales_dtype) || !value_dtype(output_dtype)) return MF_ERR_DTYPE;
    if (!expert_offsets && num_experts != 1) return MF_ERR_INVALID;
    if (rows == 0) return MF_OK;
    if (!x || !weight || !scales || !output) return MF_ERR_NULL;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(scales, 4) || !aligned(output, 4) ||
        !aligned(expert_offsets, 4) || !aligned(row_index, 4) || !aligned(zeros, 4))
        return MF_ERR_ALIGN;
    const mf::DeviceInfo *d = nullptr;
    const ExpertDevice *e = nullptr;
    mf_status st = expert_device(kInt4, &d, &e);
    if (st != MF_OK) return st;
    mf::GemvArgs a = {};
    a.x = x;
    a.x_rows = x_rows;
    a.x_ld = x_stride;
    a.row_index = row_index;
    a.w = weight;
    a.scales = scales;
    a.scale_fp32 = scales_dtype == MF_DTYPE_FP32;
    a.zeros = zeros;
    a.group = group_size;
    a.offsets = expert_offsets;
    a.rows = rows;
    a.num_experts = num_experts;
    a.n = n;
    a.k = k;
    a.out = output;
    a.out_fp32 = output_dtype == MF_DTYPE_FP32;
    a.out_ld = output_stride;
    a.num_sms = d->num_sms;
    a.status = d->status;
    a.timeout_ns = mf::kWaitLimitNs;
    a.programmatic = mf::programmatic_launch();
    return from_launch(
        mf::launch_grouped_gemv_int4(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
