"""The steps of an expert layer before the finalize: the permutation by expert,
the matrix products over each expert's rows with their gradients, and the
product with 4-bit weights.

A layer, from routed ids to the finalize's output::

    offsets, idx, row_token = mf.moe_expert_permutation(expert_ids, num_experts)
    mf.moe_grouped_gemm(tokens, w_up, offsets, up, row_index=row_token)
    act = ...                                    # the layer's activation of `up`
    mf.moe_grouped_gemm(act, w_down, offsets, down)
    mf.moe_finalize_rmsnorm(down, expert_weights, idx, norm_weight, output, ...)

and back, from the gradient of ``up``::

    mf.moe_grouped_gemm_wgrad(d_up, tokens, offsets, d_w_up, row_index=row_token)
    mf.moe_grouped_gemm_dgrad(d_up, w_up, offsets, d_rows)
    mf.moe_permuted_row_sum(d_rows, idx, d_tokens)

Like the rest of the binding this checks tensor metadata and calls the C ABI
(include/moe_finalize.h has the full contract).  The calls are asynchronous on
``stream`` (default: the current stream); values in index tensors are never
read on the host.
"""
from __future__ import annotations

from contextlib import nullcontext

import torch

from ._abi import MF_DTYPE_BF16, MF_DTYPE_FP32, check, lib
from ._binding import _on_device, _req, _stream_ptr

_BF16 = torch.bfloat16
_ROW_DTYPES = (torch.bfloat16,)
_VALUE_DTYPES = {torch.bfloat16: MF_DTYPE_BF16, torch.float32: MF_DTYPE_FP32}


def _rows(t: torch.Tensor, name: str, dtypes=_ROW_DTYPES) -> int:
    """Check a 2-D row-major operand; returns its row stride in elements."""
    if t.dim() != 2 or t.dtype not in dtypes or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be a 2-D tensor of {' or '.join(map(str, dtypes))} with "
                         "unit last-dim stride")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]  # one row: no stride to keep


def _output_rows(t: torch.Tensor, name: str) -> int:
    ld = _rows(t, name, _VALUE_DTYPES)
    if t.shape[0] > 1 and ld < t.shape[1]:
        raise ValueError(f"{name}'s rows must not overlap")
    return ld


def _index(t: torch.Tensor, name: str, shape: tuple) -> None:
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)}")


def _same_device(dev: torch.device, *tensors) -> None:
    if dev.type == "cuda":
        for t in tensors:
            if t is not None and t.device != dev:
                break
        else:
            return
    raise ValueError("all tensors must be on the same CUDA device")


def _int32(sizes: int) -> None:
    """Sizes (or-ed together) that the C interface takes as 32-bit integers: a larger one
    would lose its upper bits on the way."""
    if sizes >> 31 not in (0, -1):
        raise ValueError("a size does not fit into 32 bits")


def _ptr(t):
    return None if t is None else t.data_ptr()


def moe_expert_permutation(expert_ids: torch.Tensor, num_experts: int, *, packed: bool = False,
                           expert_offsets: torch.Tensor | None = None,
                           expanded_idx: torch.Tensor | None = None,
                           row_tokens: torch.Tensor | None = None,
                           stream: torch.cuda.Stream | None = None
                           ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Sort the routed slots by expert (stable).  Returns ``(expert_offsets,
    expanded_idx_to_permuted_idx, permuted_row_to_token)``, int32 of
    ``[num_experts + 1]``, ``[num_tokens, top_k]`` and ``[num_tokens * top_k]``.

    expert_ids: contiguous int32 [num_tokens, top_k]; with ``packed`` they are
    routing words ``(expert_id << 16) | bf16 weight bits``.  A slot whose id is
    outside [0, num_experts) gets no row: its map entry is -1, and row_to_token
    is -1 behind the last row.  The outputs are allocated unless given; they may
    not overlap the ids or each other.
    """
    _req(expert_ids.dim() == 2 and expert_ids.dtype == torch.int32 and expert_ids.is_contiguous(),
         "expert_ids must be a contiguous 2-D int32 tensor")
    dev = expert_ids.device
    T, K = expert_ids.shape
    num_experts = int(num_experts)
    _int32(K | num_experts)
    _same_device(dev, expert_offsets, expanded_idx, row_tokens)
    if expert_offsets is not None:
        _index(expert_offsets, "expert_offsets", (num_experts + 1,))
    if expanded_idx is not None:
        _index(expanded_idx, "expanded_idx", (T, K))
    if row_tokens is not None:
        _index(row_tokens, "row_tokens", (T * K,))
    # memory allocated here belongs to the stream that writes it
    with nullcontext() if stream is None else torch.cuda.stream(stream):
        if expert_offsets is None:
            expert_offsets = torch.empty(max(num_experts, 0) + 1, dtype=torch.int32, device=dev)
        if expanded_idx is None:
            expanded_idx = torch.empty((T, K), dtype=torch.int32, device=dev)
        if row_tokens is None:
            row_tokens = torch.empty(T * K, dtype=torch.int32, device=dev)
    st = _on_device(dev, lib().moe_expert_permutation, expert_ids.data_ptr(), int(bool(packed)),
                    T, K, num_experts, expert_offsets.data_ptr(), expanded_idx.data_ptr(),
                    row_tokens.data_ptr(), _stream_ptr(stream, dev))
    check(st, "moe_expert_permutation")
    return expert_offsets, expanded_idx, row_tokens


def moe_permuted_row_sum(permuted: torch.Tensor, expanded_idx: torch.Tensor, output: torch.Tensor,
                         *, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``output[t] = sum over j of permuted[expanded_idx[t, j]]`` in FP32, the
    gradient of gathering a token's row into its slots.  permuted: BF16 or FP32
    [rows, >= hidden] (unit last-dim stride, row stride a multiple of 8);
    expanded_idx: int32 [num_tokens, top_k], entries outside the rows contribute
    zero; output: contiguous BF16 or FP32 [num_tokens, hidden].  Returns it."""
    ld = _rows(permuted, "permuted", _VALUE_DTYPES)
    if output.dim() != 2 or output.dtype not in _VALUE_DTYPES or not output.is_contiguous():
        raise ValueError("output must be a contiguous 2-D BF16 or FP32 tensor")
    if expanded_idx.dim() != 2:
        raise ValueError("expanded_idx must be 2-D")
    T, hidden = output.shape
    K = expanded_idx.shape[1]
    _int32(hidden | K)
    _index(expanded_idx, "expanded_idx", (T, K))
    rows, width = permuted.shape
    if width < hidden:
        raise ValueError("permuted has fewer columns than output")
    dev = output.device
    _same_device(dev, permuted, expanded_idx)
    st = _on_device(dev, lib().moe_permuted_row_sum, permuted.data_ptr(),
                    _VALUE_DTYPES[permuted.dtype], rows, ld, expanded_idx.data_ptr(),
                    output.data_ptr(), _VALUE_DTYPES[output.dtype], T, hidden, K,
                    _stream_ptr(stream, dev))
    check(st, "moe_permuted_row_sum")
    return output


def _weight(weight: torch.Tensor, offsets: torch.Tensor) -> tuple[int, int, int, int, int]:
    """(experts, n, k, row stride, expert stride) of a [E, n, k] weight."""
    _req(weight.dim() == 3 and weight.dtype == _BF16 and
         (weight.stride(2) == 1 or weight.shape[2] <= 1),
         "weight must be a 3-D BF16 tensor with unit last-dim stride")
    E, n, k = weight.shape
    _int32(E | n | k)
    _index(offsets, "expert_offsets", (E + 1,))
    row = weight.stride(1) if n > 1 else k
    return E, n, k, row, weight.stride(0) if E > 1 else n * row


def _row_index(row_index, rows: int, x_rows: int) -> None:
    if row_index is None:
        _req(x_rows >= rows, "x has fewer rows than the product")
    else:
        _index(row_index, "row_index", (rows,))
        _req(x_rows > 0 or rows == 0, "row_index needs rows to select from")


def moe_grouped_gemm(x: torch.Tensor, weight: torch.Tensor, expert_offsets: torch.Tensor,
                     output: torch.Tensor, *, row_index: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``output[r] = weight[e] @ x[row_index[r]]`` for the rows
    ``expert_offsets[e] <= r < expert_offsets[e + 1]`` of each expert (row r of
    x without ``row_index``); rows outside every expert are left as they were.

    x: BF16 [x_rows, k]; weight: BF16 [experts, n, k]; output: BF16 or FP32
    [rows, n]; n and k multiples of 8, unit last-dim strides, other strides
    multiples of 8.  expert_offsets: int32 [experts + 1], ascending.  row_index:
    int32 [rows]; an entry outside x selects a row of zeros.  Returns ``output``.
    """
    E, n, k, w_row, w_expert = _weight(weight, expert_offsets)
    x_ld = _rows(x, "x")
    out_ld = _output_rows(output, "output")
    rows = output.shape[0]
    _req(x.shape[1] == k and output.shape[1] == n, "shapes disagree on n or k")
    _row_index(row_index, rows, x.shape[0])
    dev = output.device
    _same_device(dev, x, weight, expert_offsets, row_index)
    st = _on_device(dev, lib().moe_grouped_gemm, x.data_ptr(), x.shape[0], x_ld, _ptr(row_index),
                    weight.data_ptr(), w_row, w_expert, expert_offsets.data_ptr(),
                    output.data_ptr(), _VALUE_DTYPES[output.dtype], out_ld, rows, E, n, k,
                    _stream_ptr(stream, dev))
    check(st, "moe_grouped_gemm")
    return output


def moe_grouped_gemm_dgrad(grad_output: torch.Tensor, weight: torch.Tensor,
                           expert_offsets: torch.Tensor, grad_input: torch.Tensor, *,
                           stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Gradient of ``moe_grouped_gemm`` with respect to its rows:
    ``grad_input[r] = weight[e].T @ grad_output[r]`` (BF16 [rows, n] to BF16 or
    FP32 [rows, k]).  Rows outside every expert are left as they were.  Where the
    forward pass gathered, ``moe_permuted_row_sum`` adds the rows up per token."""
    E, n, k, w_row, w_expert = _weight(weight, expert_offsets)
    dy_ld = _rows(grad_output, "grad_output")
    dx_ld = _output_rows(grad_input, "grad_input")
    rows = grad_input.shape[0]
    _req(grad_output.shape[1] == n and grad_input.shape[1] == k and grad_output.shape[0] >= rows,
         "shapes disagree on n, k or the rows")
    dev = grad_input.device
    _same_device(dev, grad_output, weight, expert_offsets)
    st = _on_device(dev, lib().moe_grouped_gemm_dgrad, grad_output.data_ptr(), dy_ld,
                    weight.data_ptr(), w_row, w_expert, expert_offsets.data_ptr(),
                    grad_input.data_ptr(), _VALUE_DTYPES[grad_input.dtype], dx_ld, rows, E, n, k,
                    _stream_ptr(stream, dev))
    check(st, "moe_grouped_gemm_dgrad")
    return grad_input


def moe_grouped_gemm_wgrad(grad_output: torch.Tensor, x: torch.Tensor,
                           expert_offsets: torch.Tensor, grad_weight: torch.Tensor, *,
                           row_index: torch.Tensor | None = None, accumulate: bool = False,
                           stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Gradient of ``moe_grouped_gemm`` with respect to its weights:
    ``grad_weight[e] = sum over e's rows of outer(grad_output[r], x[row_index[r]])``,
    added to what ``grad_weight`` holds with ``accumulate``.  grad_weight:
    contiguous BF16 or FP32 [experts, n, k]; an expert without rows gets zeros."""
    _req(grad_weight.dim() == 3 and grad_weight.dtype in _VALUE_DTYPES and
         grad_weight.is_contiguous(), "grad_weight must be a contiguous 3-D BF16 or FP32 tensor")
    E, n, k = grad_weight.shape
    _int32(E | n | k)
    _index(expert_offsets, "expert_offsets", (E + 1,))
    dy_ld = _rows(grad_output, "grad_output")
    x_ld = _rows(x, "x")
    rows = grad_output.shape[0]
    _req(grad_output.shape[1] == n and x.shape[1] == k, "shapes disagree on n or k")
    _row_index(row_index, rows, x.shape[0])
    dev = grad_weight.device
    _same_device(dev, grad_output, x, expert_offsets, row_index)
    st = _on_device(dev, lib().moe_grouped_gemm_wgrad, grad_output.data_ptr(), dy_ld, x.data_ptr(),
                    x.shape[0], x_ld, _ptr(row_index), expert_offsets.data_ptr(),
                    grad_weight.data_ptr(), _VALUE_DTYPES[grad_weight.dtype],
                    int(bool(accumulate)), rows, E, n, k, _stream_ptr(stream, dev))
    check(st, "moe_grouped_gemm_wgrad")
    return grad_weight


def moe_grouped_gemv_int4(x: torch.Tensor, weight: torch.Tensor, scales: torch.Tensor,
                          expert_offsets: torch.Tensor | None, output: torch.Tensor, *,
                          zeros: torch.Tensor | None = None,
                          row_index: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``moe_grouped_gemm`` with 4-bit weights, for few rows per expert.

    weight: contiguous uint8 [experts, n, k / 2], column c in the low half of
    byte c / 2 for even c, in the high half for odd c.  scales: contiguous BF16
    or FP32 [experts, n, k / group] with a group of 32, 64 or 128 columns; zeros:
    contiguous uint8 of the same shape (0..15), or None for 8 everywhere.  A
    weight is ``(q - zero) * scale``.  x: BF16 [x_rows, k]; output: BF16 or FP32
    [rows, n].  expert_offsets None (one expert only): every row belongs to the
    one matrix.  Returns ``output``.
    """
    _req(weight.dim() == 3 and weight.dtype == torch.uint8 and weight.is_contiguous(),
         "weight must be a contiguous 3-D uint8 tensor")
    E, n, k = weight.shape[0], weight.shape[1], 2 * weight.shape[2]
    _int32(E | n | k)
    _req(scales.dim() == 3 and scales.dtype in _VALUE_DTYPES and scales.is_contiguous() and
         scales.shape[:2] == (E, n), "scales must be contiguous BF16 or FP32 [experts, n, groups]")
    groups = scales.shape[2]
    _req(groups > 0 and k % groups == 0 and k // groups in (32, 64, 128),
         "scales must cover groups of 32, 64 or 128 columns")
    _req(zeros is None or (zeros.dtype == torch.uint8 and zeros.shape == scales.shape and
                           zeros.is_contiguous()),
         "zeros must be a contiguous uint8 tensor of the scales' shape")
    if expert_offsets is None:
        _req(E == 1, "expert_offsets may be None with one expert only")
    else:
        _index(expert_offsets, "expert_offsets", (E + 1,))
    x_ld = _rows(x, "x")
    out_ld = _output_rows(output, "output")
    rows = output.shape[0]
    _req(x.shape[1] == k and output.shape[1] == n, "shapes disagree on n or k")
    _row_index(row_index, rows, x.shape[0])
    dev = output.device
    _same_device(dev, x, weight, scales, expert_offsets, zeros, row_index)
    st = _on_device(dev, lib().moe_grouped_gemv_int4, x.data_ptr(), x.shape[0], x_ld,
                    _ptr(row_index), weight.data_ptr(), scales.data_ptr(),
                    _VALUE_DTYPES[scales.dtype], _ptr(zeros), k // groups, _ptr(expert_offsets),
                    output.data_ptr(), _VALUE_DTYPES[output.dtype], out_ld, rows, E, n, k,
                    _stream_ptr(stream, dev))
    check(st, "moe_grouped_gemv_int4")
    return output
