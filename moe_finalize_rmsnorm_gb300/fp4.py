"""Microscaled 4-bit floating point: rows to 4 bits and back, and the expert layer's
product of 4-bit rows with 4-bit weights.

Values are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte (uint8,
the even column in the low half), and a block of columns shares a scale.  The scales' dtype
names the format: ``torch.float8_e8m0fnu`` are powers of two over blocks of 32 columns,
``torch.float8_e4m3fn`` are E4M3 over blocks of 16 (their signs are not used).  Rows of
bytes and of scales begin at multiples of 16 bytes; ``moe_fp4_empty`` allocates such
pairs::

    q, scales = mf.moe_fp4_empty((num_tokens,), hidden, torch.float8_e4m3fn)
    mf.moe_quantize_fp4(tokens, q, scales)
    mf.moe_grouped_gemm_fp4(q, scales, w, w_scales, offsets, up, row_index=row_token)

Like the rest of the binding this checks tensor metadata and calls the C ABI
(include/moe_finalize.h has the full contract).
"""
from __future__ import annotations

from contextlib import nullcontext

import torch

from ._abi import MF_FP4_MX, MF_FP4_NV, check, lib
from ._binding import _on_device, _req, _stream_ptr
from .combine import _matrix
from .experts import _index, _int32, _ptr, _row_index, _same_device

_FORMATS = {torch.float8_e8m0fnu: (MF_FP4_MX, 32), torch.float8_e4m3fn: (MF_FP4_NV, 16)}


def moe_fp4_empty(shape: tuple, k: int, scale_dtype: torch.dtype, *, device="cuda",
                  stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Uninitialised ``(quantized [*shape, k / 2], scales [*shape, k / block])`` whose rows
    begin at multiples of 16 bytes."""
    _req(scale_dtype in _FORMATS, f"the scales' dtype must be one of {list(_FORMATS)}")
    k = int(k)
    _req(k > 0 and k % 32 == 0, "k must be a multiple of 32")
    groups = k // _FORMATS[scale_dtype][1]
    with nullcontext() if stream is None else torch.cuda.stream(stream):
        q = torch.empty((*shape, k // 2), dtype=torch.uint8, device=device)
        s = torch.empty((*shape, (groups + 15) // 16 * 16), dtype=torch.uint8, device=device)
    return q, s[..., :groups].view(scale_dtype)


def _packed(q: torch.Tensor, scales: torch.Tensor, name: str, dims: int
            ) -> tuple[int, int, int, int]:
    """Check packed values and their scales; returns (format, k, bytes between the rows of
    the values and of the scales)."""
    qn, qst = q.shape, q.stride()
    if len(qn) != dims or q.dtype != torch.uint8 or (qst[-1] != 1 and qn[-1] > 1):
        raise ValueError(f"{name} must be a {dims}-D uint8 tensor with unit last-dim stride")
    f = _FORMATS.get(scales.dtype)
    sn, sst = scales.shape, scales.stride()
    if f is None or len(sn) != dims or (sst[-1] != 1 and sn[-1] > 1):
        raise ValueError(f"{name}'s scales must be a {dims}-D tensor of float8_e8m0fnu or "
                         "float8_e4m3fn with unit last-dim stride")
    width, groups = qn[-1], sn[-1]
    if width % 16 != 0 or sn[:-1] != qn[:-1] or groups * f[1] != 2 * width:
        raise ValueError(f"{name}'s scales must cover blocks of {f[1]} columns of its rows, "
                         "and its columns must be a multiple of 32")
    if qn[-2] > 1:
        return f[0], 2 * width, qst[-2], sst[-2]
    return f[0], 2 * width, width, (groups + 15) // 16 * 16  # one row: no stride to keep


def _whole_pieces(scales: torch.Tensor, name: str, behind: int) -> None:
    """The product reads scales in 16-byte pieces: the last row's has to lie in its memory."""
    if scales.numel() == 0:
        return
    end = scales.storage_offset() + 1 + behind
    for n, st in zip(scales.shape, scales.stride()):
        end += (n - 1) * st
    if end > scales.untyped_storage().nbytes():
        raise ValueError(f"{name}'s last row must be followed by bytes up to a multiple of 16 "
                         "(as moe_fp4_empty allocates)")


def moe_quantize_fp4(x: torch.Tensor, quantized: torch.Tensor, scales: torch.Tensor, *,
                     factor: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None
                     ) -> tuple[torch.Tensor, torch.Tensor]:
    """Rows to 4-bit floating point.  Of a block of ``v = factor * x`` with largest
    magnitude m the scale is ``2 ** (floor(log2(m)) - 2)`` (E8M0) or ``m / 6`` rounded to
    E4M3, at most 448; a value is the nearest E2M1 of ``v / scale``, ties to even, at most 6
    in magnitude, and 0 where the scale is 0.  A block that holds an infinity or a NaN gets
    a NaN scale and zeros.

    x: BF16 or FP32 [rows, k], unit last-dim stride, row stride a multiple of 8, k a
    multiple of 32; factor: FP32 tensor of one element.  Returns ``(quantized, scales)``.
    """
    rows, width, x_ld, x_dtype = _matrix(x, "x")
    fmt, k, q_ld, s_ld = _packed(quantized, scales, "quantized", 2)
    _req(2 * q_ld >= k and s_ld * 32 >= k, "the rows of quantized and scales must not overlap")
    _req(quantized.shape[0] == rows and k == width,
         "x and quantized disagree on the rows or on k")
    _req(factor is None or (factor.dtype == torch.float32 and factor.numel() == 1),
         "factor must be an FP32 tensor of one element")
    _int32(k)
    dev = quantized.device
    _same_device(dev, x, scales, factor)
    st = _on_device(dev, lib().moe_quantize_fp4, x.data_ptr(), x_dtype, x_ld,
                    _ptr(factor), quantized.data_ptr(), q_ld, scales.data_ptr(), s_ld, fmt, rows,
                    k, _stream_ptr(stream, dev))
    check(st, "moe_quantize_fp4")
    return quantized, scales


def moe_dequantize_fp4(quantized: torch.Tensor, scales: torch.Tensor, output: torch.Tensor, *,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """What 4-bit values stand for: ``output = value * scale`` (exact in FP32; in BF16 too,
    but for values beyond its range).  output: BF16 or FP32 [rows, k], unit last-dim
    stride, row stride a multiple of 8.  Returns ``output``."""
    fmt, k, q_ld, s_ld = _packed(quantized, scales, "quantized", 2)
    rows, width, out_ld, out_dtype = _matrix(output, "output", written=True)
    _req(quantized.shape[0] == rows and k == width,
         "output and quantized disagree on the rows or on k")
    _int32(k)
    dev = output.device
    _same_device(dev, quantized, scales)
    st = _on_device(dev, lib().moe_dequantize_fp4, quantized.data_ptr(), q_ld,
                    scales.data_ptr(), s_ld, fmt, output.data_ptr(), out_dtype, out_ld, rows, k,
                    _stream_ptr(stream, dev))
    check(st, "moe_dequantize_fp4")
    return output


def moe_grouped_gemm_fp4(x: torch.Tensor, x_scales: torch.Tensor, weight: torch.Tensor,
                         weight_scales: torch.Tensor, expert_offsets: torch.Tensor | None,
                         output: torch.Tensor, *, row_index: torch.Tensor | None = None,
                         factor: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``moe_grouped_gemm`` of 4-bit rows with 4-bit weights, both of one format:
    ``output[r] = factor[e] * (weight[e] @ x[row_index[r]])`` for each expert's rows, other
    rows left as they were.

    x: uint8 [x_rows, k / 2] and its scales; weight: uint8 [experts, n, k / 2] and its scales;
    output: BF16 or FP32 [rows, n], not over an input; n a multiple of 8, k of 32.  factor: contiguous FP32
    [experts], or None.  expert_offsets: int32 [experts + 1], ascending, or None (one
    expert only): every row belongs to the one matrix.  row_index: int32 [rows]; an entry
    outside x selects a row of zeros.  Returns ``output``.
    """
    fmt, k, w_ld, ws_ld = _packed(weight, weight_scales, "weight", 3)
    x_fmt, x_k, x_ld, xs_ld = _packed(x, x_scales, "x", 2)
    _req(x_fmt == fmt, "x and weight must have one format")
    E, n, _ = weight.shape
    rows, out_n, out_ld, out_dtype = _matrix(output, "output", written=True)
    x_rows = x.shape[0]
    _req(x_k == k and out_n == n, "shapes disagree on n or k")
    _int32(E | n | k)
    if expert_offsets is None:
        _req(E == 1, "expert_offsets may be None with one expert only")
    else:
        _index(expert_offsets, "expert_offsets", (E + 1,))
    _row_index(row_index, rows, x_rows)
    behind = -(k // (32 if fmt == MF_FP4_MX else 16)) % 16  # bytes up to a whole piece
    if behind:
        _whole_pieces(x_scales, "x", behind)
        _whole_pieces(weight_scales, "weight", behind)
    _req(factor is None or (factor.dtype == torch.float32 and factor.shape == (E,) and
                            factor.is_contiguous()), "factor must be contiguous FP32 [experts]")
    dev = output.device
    _same_device(dev, x, x_scales, weight, weight_scales, expert_offsets, row_index, factor)
    st = _on_device(dev, lib().moe_grouped_gemm_fp4, x.data_ptr(), x_rows, x_ld,
                    x_scales.data_ptr(), xs_ld, _ptr(row_index), weight.data_ptr(), w_ld,
                    weight.stride(0), weight_scales.data_ptr(), ws_ld, weight_scales.stride(0),
                    fmt, _ptr(factor), _ptr(expert_offsets), output.data_ptr(),
                    out_dtype, out_ld, rows, E, n, k, _stream_ptr(stream, dev))
    check(st, "moe_grouped_gemm_fp4")
    return output
