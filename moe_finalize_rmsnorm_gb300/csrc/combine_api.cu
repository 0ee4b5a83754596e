// C ABI of the way into expert order and back: argument validation and launches.
// Declarations and the contract are in include/moe_finalize.h.
#include <cuda_runtime.h>

#include "checks.h"
#include "device_info.h"
#include "experts.h"
#include "moe_finalize.h"

namespace {

using mf::aligned;

int value_bytes(mf_dtype d) { return d == MF_DTYPE_FP32 ? 4 : 2; }

// Bytes from the first element of strided rows to the last.
int64_t extent(int64_t rows, int64_t stride, int32_t hidden, mf_dtype d) {
    return rows > 0 ? ((rows - 1) * stride + hidden) * value_bytes(d) : 0;
}

mf_status check_sizes(int64_t num_tokens, int64_t rows, int32_t hidden, int32_t top_k) {
    if (hidden < 8 || hidden > mf::kMaxWidth || hidden % 8 != 0 || top_k < 1 || top_k > 32)
        return MF_ERR_UNSUPPORTED;
    if (rows < 0 || rows > mf::kMaxRows || num_tokens < 0 || num_tokens > mf::kMaxRows / top_k)
        return MF_ERR_SHAPE;
    // a thread for every four columns, 128 to a block
    if ((num_tokens * (hidden / 4) + 127) / 128 > 0x7fffffffLL) return MF_ERR_SHAPE;
    return MF_OK;
}

bool weight_dtype(mf_dtype d) {
    return d == MF_DTYPE_BF16 || d == MF_DTYPE_FP32 || d == MF_DTYPE_PACKED_TOPK;
}

mf_status start(mf::CombineArgs &a, const int32_t *idx, const void *weights, mf_dtype weights_dtype,
                int64_t rows, int64_t num_tokens, int32_t hidden, int32_t top_k) {
    const mf::DeviceInfo *d = nullptr;
    const mf_status st = mf::device_info(&d);
    if (st != MF_OK) return st;
    static_assert(int{MF_DTYPE_BF16} == mf::kRoutingBf16 && int{MF_DTYPE_FP32} == mf::kRoutingFp32 &&
                      int{MF_DTYPE_PACKED_TOPK} == mf::kRoutingPacked,
                  "the kernels' weight kinds");
    a.idx = idx;
    a.weights = weights;
    a.weight_kind = weights ? static_cast<int>(weights_dtype) : mf::kRoutingNone;
    a.num_rows = rows;
    a.num_tokens = num_tokens;
    a.hidden = hidden;
    a.top_k = top_k;
    a.num_sms = d->num_sms;
    a.programmatic = mf::programmatic_launch();
    return MF_OK;
}

}  // namespace

extern "C" {

mf_status moe_dispatch(const void *x, mf_dtype x_dtype, int64_t x_stride,
                       const void *expert_weights, mf_dtype weights_dtype,
                       const int32_t *expanded_idx_to_permuted_idx, void *output,
                       mf_dtype output_dtype, int64_t rows, int64_t output_stride,
                       int64_t num_tokens, int32_t hidden, int32_t top_k, mf_stream_t stream) {
    mf_status st = check_sizes(num_tokens, rows, hidden, top_k);
    if (st != MF_OK) return st;
    if (!mf::row_stride_ok(x_stride, hidden) || !mf::row_stride_ok(output_stride, hidden))
        return MF_ERR_SHAPE;
    if (!mf::value_dtype(x_dtype) || !mf::value_dtype(output_dtype) ||
        (expert_weights && !weight_dtype(weights_dtype)))
        return MF_ERR_DTYPE;
    if (num_tokens == 0 || rows == 0) return MF_OK;
    if (!x || !expanded_idx_to_permuted_idx || !output) return MF_ERR_NULL;
    if (!aligned(x, 16) || !aligned(output, 16) || !aligned(expanded_idx_to_permuted_idx, 4) ||
        !aligned(expert_weights, weights_dtype == MF_DTYPE_BF16 ? 2 : 4))
        return MF_ERR_ALIGN;
    const int64_t out_bytes = extent(rows, output_stride, hidden, output_dtype);
    const int64_t slots = num_tokens * top_k;
    if (mf::overlap(output, out_bytes, x, extent(num_tokens, x_stride, hidden, x_dtype)) ||
        mf::overlap(output, out_bytes, expanded_idx_to_permuted_idx, 4 * slots) ||
        (expert_weights && mf::overlap(output, out_bytes, expert_weights,
                                       slots * (weights_dtype == MF_DTYPE_BF16 ? 2 : 4))))
        return MF_ERR_ALIGN;
    mf::CombineArgs a = {};
    st = start(a, expanded_idx_to_permuted_idx, expert_weights, weights_dtype, rows, num_tokens,
               hidden, top_k);
    if (st != MF_OK) return st;
    a.token_rows = x;
    a.token_ld = x_stride;
    a.token_fp32 = x_dtype == MF_DTYPE_FP32;
    a.rows_fp32 = output_dtype == MF_DTYPE_FP32;
    a.out_rows = output;
    a.out_ld = output_stride;
    return mf::from_launch(mf::launch_dispatch(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_combine(const void *permuted, mf_dtype permuted_dtype, int64_t rows,
                      int64_t row_stride, const void *expert_weights, mf_dtype weights_dtype,
                      const int32_t *expanded_idx_to_permuted_idx, void *output,
                      mf_dtype output_dtype, int64_t output_stride, int64_t num_tokens,
                      int32_t hidden, int32_t top_k, mf_stream_t stream) {
    mf_status st = check_sizes(num_tokens, rows, hidden, top_k);
    if (st != MF_OK) return st;
    if (!mf::row_stride_ok(row_stride, hidden) || !mf::row_stride_ok(output_stride, hidden))
        return MF_ERR_SHAPE;
    if (!mf::value_dtype(permuted_dtype) || !mf::value_dtype(output_dtype) ||
        !weight_dtype(weights_dtype))
        return MF_ERR_DTYPE;
    if (num_tokens == 0) return MF_OK;
    if (!expert_weights || !expanded_idx_to_permuted_idx || !output || (rows > 0 && !permuted))
        return MF_ERR_NULL;
    const int weight_bytes = weights_dtype == MF_DTYPE_BF16 ? 2 : 4;
    if (!aligned(permuted, 16) || !aligned(output, 16) ||
        !aligned(expanded_idx_to_permuted_idx, 4) || !aligned(expert_weights, weight_bytes))
        return MF_ERR_ALIGN;
    const int64_t out_bytes = extent(num_tokens, output_stride, hidden, output_dtype);
    const int64_t slots = num_tokens * top_k;
    if (mf::overlap(output, out_bytes, permuted, extent(rows, row_stride, hidden, permuted_dtype)) ||
        mf::overlap(output, out_bytes, expanded_idx_to_permuted_idx, 4 * slots) ||
        mf::overlap(output, out_bytes, expert_weights, slots * weight_bytes))
        return MF_ERR_ALIGN;
    mf::CombineArgs a = {};
    st = start(a, expanded_idx_to_permuted_idx, expert_weights, weights_dtype, rows, num_tokens,
               hidden, top_k);
    if (st != MF_OK) return st;
    a.rows = permuted;
    a.ld = row_stride;
    a.rows_fp32 = permuted_dtype == MF_DTYPE_FP32;
    a.token_fp32 = output_dtype == MF_DTYPE_FP32;
    a.out_rows = output;
    a.out_ld = output_stride;
    return mf::from_launch(mf::launch_combine(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_combine_backward(const void *grad_output, mf_dtype grad_output_dtype,
                               int64_t grad_output_stride, const void *permuted,
                               mf_dtype permuted_dtype, int64_t rows, int64_t row_stride,
                               const void *expert_weights, mf_dtype weights_dtype,
                               const int32_t *expanded_idx_to_permuted_idx, void *grad_permuted,
                               int64_t grad_permuted_stride, void *grad_weights,
                               mf_dtype grad_weights_dtype, int64_t num_tokens, int32_t hidden,
                               int32_t top_k, mf_stream_t stream) {
    mf_status st = check_sizes(num_tokens, rows, hidden, top_k);
    if (st != MF_OK) return st;
    if (!mf::row_stride_ok(grad_output_stride, hidden) ||
        (grad_weights && !mf::row_stride_ok(row_stride, hidden)) ||
        (grad_permuted && !mf::row_stride_ok(grad_permuted_stride, hidden)))
        return MF_ERR_SHAPE;
    if (!mf::value_dtype(grad_output_dtype) || !mf::value_dtype(permuted_dtype) ||
        (grad_permuted && !weight_dtype(weights_dtype)) ||
        (grad_weights && !mf::value_dtype(grad_weights_dtype)))
        return MF_ERR_DTYPE;
    if (num_tokens == 0) return MF_OK;
    // (without rows a gradient of theirs may be a null pointer, as that of an empty tensor)
    if (!grad_permuted && !grad_weights && rows > 0) return MF_ERR_INVALID;
    if (!grad_output || !expanded_idx_to_permuted_idx || (grad_permuted && !expert_weights) ||
        (grad_weights && rows > 0 && !permuted))
        return MF_ERR_NULL;
    const int weight_bytes = weights_dtype == MF_DTYPE_BF16 ? 2 : 4;
    if (!aligned(grad_output, 16) || (grad_weights && !aligned(permuted, 16)) ||
        !aligned(grad_permuted, 16) || !aligned(expanded_idx_to_permuted_idx, 4) ||
        (grad_permuted && !aligned(expert_weights, weight_bytes)) ||
        (grad_weights && !aligned(grad_weights, value_bytes(grad_weights_dtype))))
        return MF_ERR_ALIGN;
    const int64_t slots = num_tokens * top_k;
    const struct {
        const void *p;
        int64_t bytes;
    } in[4] = {{grad_output, extent(num_tokens, grad_output_stride, hidden, grad_output_dtype)},
               {permuted, grad_weights ? extent(rows, row_stride, hidden, permuted_dtype) : 0},
               {expert_weights, grad_permuted ? slots * weight_bytes : 0},
               {expanded_idx_to_permuted_idx, 4 * slots}};
    const int64_t rows_bytes =
        grad_permuted ? extent(rows, grad_permuted_stride, hidden, permuted_dtype) : 0;
    const int64_t weights_bytes = grad_weights ? slots * value_bytes(grad_weights_dtype) : 0;
    for (const auto &i : in)
        if (mf::overlap(grad_permuted, rows_bytes, i.p, i.bytes) ||
            mf::overlap(grad_weights, weights_bytes, i.p, i.bytes))
            return MF_ERR_ALIGN;
    if (mf::overlap(grad_permuted, rows_bytes, grad_weights, weights_bytes)) return MF_ERR_ALIGN;
    if (rows == 0 && !grad_weights) return MF_OK;
    mf::CombineArgs a = {};
    st = start(a, expanded_idx_to_permuted_idx, expert_weights, weights_dtype, rows, num_tokens,
               hidden, top_k);
    if (st != MF_OK) return st;
    a.token_rows = grad_output;
    a.token_ld = grad_output_stride;
    a.token_fp32 = grad_output_dtype == MF_DTYPE_FP32;
    a.rows = permuted;
    a.ld = row_stride;
    a.rows_fp32 = permuted_dtype == MF_DTYPE_FP32;
    a.out_rows = grad_permuted;
    a.out_ld = grad_permuted_stride;
    a.grad_weights = grad_weights;
    a.grad_weights_fp32 = grad_weights_dtype == MF_DTYPE_FP32;
    return mf::from_launch(mf::launch_combine_backward(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
