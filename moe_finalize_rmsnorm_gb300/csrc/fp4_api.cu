// C ABI of the 4-bit floating point operations: argument validation and launches.
// Declarations and the contract are in include/moe_finalize.h.
#include <cuda_runtime.h>

#include <mutex>

#include "checks.h"
#include "device_info.h"
#include "experts.h"
#include "fp4.h"
#include "moe_finalize.h"

namespace {

using mf::aligned;

int block_of(mf_fp4_format f) { return f == MF_FP4_MX ? 32 : 16; }

bool format_ok(mf_fp4_format f) { return f == MF_FP4_MX || f == MF_FP4_NV; }

// Byte strides of packed rows and of scales: at least the row, a multiple of 16.
bool byte_stride_ok(int64_t stride, int64_t width) {
    return stride >= width && stride % 16 == 0 && stride < (int64_t{1} << 36);
}

// Scales' rows, in 32 bits, too.
bool scale_stride_ok(int64_t stride, int64_t width) {
    return byte_stride_ok(stride, width) && stride < (int64_t{1} << 31);
}

bool k_ok(int32_t k) { return k >= 32 && k <= mf::kMaxWidth && k % 32 == 0; }

int64_t extent(int64_t rows, int64_t stride, int64_t width) {
    return rows > 0 ? (rows - 1) * stride + width : 0;
}

// Experts' matrices as rows of one stride, where the experts lie a multiple of it apart.
mf::ByteRows matrices(const void *p, int64_t experts, int64_t expert_stride, int64_t n,
                      int64_t row_stride, int64_t width) {
    if (experts == 1) return {p, n, row_stride, width};
    if (expert_stride % row_stride == 0)
        return {p, (experts - 1) * (expert_stride / row_stride) + n, row_stride, width};
    return {p, 1, 0, (experts - 1) * expert_stride + extent(n, row_stride, width)};
}

mf_status check_rows(mf_fp4_format format, int64_t rows, int32_t k, mf_dtype dtype,
                     int64_t row_stride, int64_t q_stride, int64_t s_stride) {
    if (!format_ok(format)) return MF_ERR_INVALID;
    if (!k_ok(k)) return MF_ERR_UNSUPPORTED;
    if (rows < 0 || rows > mf::kMaxRows || !mf::row_stride_ok(row_stride, k) ||
        !byte_stride_ok(q_stride, k / 2) || !scale_stride_ok(s_stride, k / block_of(format)))
        return MF_ERR_SHAPE;
    // a thread for every 32 values, 128 to a block
    if ((rows * (k / 8) + 511) / 512 > 0x7fffffffLL) return MF_ERR_SHAPE;
    return mf::value_dtype(dtype) ? MF_OK : MF_ERR_DTYPE;
}

// The products' kernels are set up on the first call on a device.
struct Fp4Device {
    bool ready = false;
    int num_pairs = 0;  // resident pairs of SMs
};

constexpr int kMaxDevices = 64;
std::mutex g_fp4_mutex;
Fp4Device g_fp4_devices[kMaxDevices];

mf_status fp4_device(const mf::DeviceInfo **info, int *num_pairs) {
    const mf_status st = mf::device_info(info);
    if (st != MF_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MF_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_fp4_mutex);
    Fp4Device &d = g_fp4_devices[dev];
    if (!d.ready) {
        cudaError_t e = mf::prepare_fp4_rows();
        if (e == cudaSuccess) e = mf::prepare_fp4_gemm(&d.num_pairs);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return MF_ERR_CUDA;
        }
        d.ready = true;
    }
    *num_pairs = d.num_pairs;
    return MF_OK;
}

}  // namespace

extern "C" {

mf_status moe_quantize_fp4(const void *x, mf_dtype x_dtype, int64_t x_stride, const float *factor,
                           uint8_t *quantized, int64_t quantized_stride, uint8_t *scales,
                           int64_t scales_stride, mf_fp4_format format, int64_t rows, int32_t k,
                           mf_stream_t stream) {
    mf_status st = check_rows(format, rows, k, x_dtype, x_stride, quantized_stride, scales_stride);
    if (st != MF_OK) return st;
    if (rows == 0) return MF_OK;
    if (!x || !quantized || !scales) return MF_ERR_NULL;
    if (!aligned(x, 16) || !aligned(quantized, 16) || !aligned(scales, 16) || !aligned(factor, 4))
        return MF_ERR_ALIGN;
    const int64_t x_bytes = extent(rows, x_stride, k) * (x_dtype == MF_DTYPE_FP32 ? 4 : 2);
    const int64_t q_bytes = extent(rows, quantized_stride, k / 2);
    const int64_t s_bytes = extent(rows, scales_stride, k / block_of(format));
    if (mf::overlap(quantized, q_bytes, x, x_bytes) || mf::overlap(scales, s_bytes, x, x_bytes) ||
        mf::overlap(quantized, q_bytes, scales, s_bytes) ||
        (factor && (mf::overlap(quantized, q_bytes, factor, 4) ||
                    mf::overlap(scales, s_bytes, factor, 4))))
        return MF_ERR_ALIGN;
    const mf::DeviceInfo *d = nullptr;
    st = mf::device_info(&d);
    if (st != MF_OK) return st;
    mf::Fp4RowsArgs a = {};
    a.x = x;
    a.x_ld = x_stride;
    a.x_fp32 = x_dtype == MF_DTYPE_FP32;
    a.factor = factor;
    a.q = quantized;
    a.q_ld = quantized_stride;
    a.scales = scales;
    a.s_ld = scales_stride;
    a.format = format;
    a.rows = rows;
    a.k = k;
    a.programmatic = mf::programmatic_launch();
    return mf::from_launch(mf::launch_quantize_fp4(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_dequantize_fp4(const uint8_t *quantized, int64_t quantized_stride,
                             const uint8_t *scales, int64_t scales_stride, mf_fp4_format format,
                             void *output, mf_dtype output_dtype, int64_t output_stride,
                             int64_t rows, int32_t k, mf_stream_t stream) {
    mf_status st =
        check_rows(format, rows, k, output_dtype, output_stride, quantized_stride, scales_stride);
    if (st != MF_OK) return st;
    if (rows == 0) return MF_OK;
    if (!quantized || !scales || !output) return MF_ERR_NULL;
    if (!aligned(output, 16) || !aligned(quantized, 16) || !aligned(scales, 16))
        return MF_ERR_ALIGN;
    const int64_t out_bytes =
        extent(rows, output_stride, k) * (output_dtype == MF_DTYPE_FP32 ? 4 : 2);
    if (mf::overlap(output, out_bytes, quantized, extent(rows, quantized_stride, k / 2)) ||
        mf::overlap(output, out_bytes, scales, extent(rows, scales_stride, k / block_of(format))))
        return MF_ERR_ALIGN;
    const mf::DeviceInfo *d = nullptr;
    st = mf::device_info(&d);
    if (st != MF_OK) return st;
    mf::Fp4RowsArgs a = {};
    a.q = const_cast<uint8_t *>(quantized);
    a.q_ld = quantized_stride;
    a.scales = const_cast<uint8_t *>(scales);
    a.s_ld = scales_stride;
    a.out = output;
    a.out_ld = output_stride;
    a.out_fp32 = output_dtype == MF_DTYPE_FP32;
    a.format = format;
    a.rows = rows;
    a.k = k;
    a.programmatic = mf::programmatic_launch();
    return mf::from_launch(mf::launch_dequantize_fp4(a, reinterpret_cast<cudaStream_t>(stream)));
}

mf_status moe_grouped_gemm_fp4(const uint8_t *x, int64_t x_rows, int64_t x_stride,
                               const uint8_t *x_scales, int64_t x_scales_stride,
                               const int32_t *row_index, const uint8_t *weight,
                               int64_t weight_row_stride, int64_t weight_expert_stride,
                               const uint8_t *weight_scales, int64_t weight_scales_row_stride,
                               int64_t weight_scales_expert_stride, mf_fp4_format format,
                               const float *factor, const int32_t *expert_offsets, void *output,
                               mf_dtype output_dtype, int64_t output_stride, int64_t rows,
                               int32_t num_experts, int32_t n, int32_t k, mf_stream_t stream) {
    if (!format_ok(format)) return MF_ERR_INVALID;
    if (num_experts < 1 || num_experts > mf::kMaxExperts || n < 8 || n > mf::kMaxWidth ||
        n % 8 != 0 || !k_ok(k))
        return MF_ERR_UNSUPPORTED;
    if (rows < 0 || rows > mf::kMaxRows || x_rows < 0 || x_rows > mf::kMaxRows ||
        x_rows < (row_index ? (rows > 0) : rows))
        return MF_ERR_SHAPE;
    const int32_t groups = k / block_of(format);
    if (!byte_stride_ok(x_stride, k / 2) || !scale_stride_ok(x_scales_stride, groups) ||
        !byte_stride_ok(weight_row_stride, k / 2) ||
        !scale_stride_ok(weight_scales_row_stride, groups) ||
        !mf::row_stride_ok(output_stride, n))
        return MF_ERR_SHAPE;
    if (num_experts > 1 &&
        (!byte_stride_ok(weight_expert_stride, extent(n, weight_row_stride, k / 2)) ||
         !byte_stride_ok(weight_scales_expert_stride, extent(n, weight_scales_row_stride, groups))))
        return MF_ERR_SHAPE;
    if (!mf::value_dtype(output_dtype)) return MF_ERR_DTYPE;
    if (!expert_offsets && num_experts != 1) return MF_ERR_INVALID;
    if (rows == 0) return MF_OK;
    if (!x || !x_scales || !weight || !weight_scales || !output) return MF_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_scales, 16) || !aligned(weight, 16) ||
        !aligned(weight_scales, 16) || !aligned(output, 16) || !aligned(expert_offsets, 4) ||
        !aligned(row_index, 4) || !aligned(factor, 4))
        return MF_ERR_ALIGN;
    const int value = output_dtype == MF_DTYPE_FP32 ? 4 : 2;
    const mf::ByteRows out = {output, rows, output_stride * value, int64_t{n} * value};
    const int64_t experts = num_experts;
    const mf::ByteRows in[7] = {
        {x, x_rows, x_stride, k / 2},
        {x_scales, x_rows, x_scales_stride, groups},
        matrices(weight, experts, weight_expert_stride, n, weight_row_stride, k / 2),
        matrices(weight_scales, experts, weight_scales_expert_stride, n, weight_scales_row_stride,
                 groups),
        {row_index, row_index ? 1 : 0, 0, 4 * rows},
        {factor, factor ? 1 : 0, 0, 4 * experts},
        {expert_offsets, expert_offsets ? 1 : 0, 0, 4 * (experts + 1)}};
    for (const mf::ByteRows &i : in)
        if (mf::overlap(out, i)) return MF_ERR_ALIGN;
    const mf::DeviceInfo *d = nullptr;
    mf::Fp4GemmArgs a = {};
    const mf_status st = fp4_device(&d, &a.num_pairs);
    if (st != MF_OK) return st;
    a.x = x;
    a.x_rows = x_rows;
    a.x_ld = x_stride;
    a.x_scales = x_scales;
    a.xs_ld = x_scales_stride;
    a.row_index = row_index;
    a.w = weight;
    a.w_ld = weight_row_stride;
    a.w_expert = num_experts > 1 ? weight_expert_stride : weight_row_stride;  // not used by one
    a.w_scales = weight_scales;
    a.ws_ld = weight_scales_row_stride;
    a.ws_expert = num_experts > 1 ? weight_scales_expert_stride : 0;
    a.factor = factor;
    a.offsets = expert_offsets;
    a.format = format;
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
    return mf::from_launch(mf::launch_fp4_gemm(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
