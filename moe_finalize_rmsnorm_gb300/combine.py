"""The tokens' rows into expert order and back, with the routing weights, and the
gradients::

    offsets, idx, row_token = mf.moe_expert_permutation(expert_ids, num_experts)
    mf.moe_dispatch(tokens, idx, rows)                    # rows in expert order
    ...                                                   # the experts: rows to `down`
    mf.moe_combine(down, expert_weights, idx, output)     # back to the tokens, weighted

and back, from the gradient of ``output``::

    mf.moe_combine_backward(d_output, down, expert_weights, idx, d_down, d_weights)
    ...                                                   # the experts: d_down to d_rows
    mf.moe_permuted_row_sum(d_rows, idx, d_tokens)

``moe_combine`` is the finalize without its norm.  Where the weights are applied on the
way in instead (``moe_dispatch`` with ``expert_weights``), the gradients of the tokens and
of the weights are::

    mf.moe_combine(d_rows, expert_weights, idx, d_tokens)
    mf.moe_combine_backward(tokens, d_rows, expert_weights, idx, None, d_weights)

Like the rest of the binding this checks tensor metadata and calls the C ABI
(include/moe_finalize.h has the full contract); values in index tensors are never read
on the host.
"""
from __future__ import annotations

import torch

from ._abi import MF_DTYPE_BF16, MF_DTYPE_FP32, MF_DTYPE_PACKED_TOPK, check, lib
from ._binding import _on_device, _req, _stream_ptr
from .experts import _VALUE_DTYPES, _int32, _ptr, _same_device

_WEIGHT_DTYPES = {torch.bfloat16: MF_DTYPE_BF16, torch.float32: MF_DTYPE_FP32,
                  torch.int32: MF_DTYPE_PACKED_TOPK}


def _matrix(t: torch.Tensor, name: str, written: bool = False) -> tuple[int, int, int, int]:
    """Check a 2-D row-major BF16 or FP32 operand; returns (rows, columns, row stride in
    elements, dtype code)."""
    shape, code = t.shape, _VALUE_DTYPES.get(t.dtype)
    if len(shape) == 2 and code is not None:
        rows, width = shape
        ld, unit = t.stride()
        if unit == 1 or width <= 1:
            if rows <= 1:
                return rows, width, (width + 7) // 8 * 8, code  # one row: no stride to keep
            if written and ld < width:
                raise ValueError(f"{name}'s rows must not overlap")
            return rows, width, ld, code
    raise ValueError(f"{name} must be a 2-D BF16 or FP32 tensor with unit last-dim stride")


def _slots(expanded_idx: torch.Tensor, expert_weights) -> tuple[int, int, int]:
    """(tokens, top_k, the weights' dtype code) of a map and its weights."""
    shape = expanded_idx.shape
    if len(shape) != 2 or expanded_idx.dtype != torch.int32 or not expanded_idx.is_contiguous():
        raise ValueError("expanded_idx must be a contiguous 2-D int32 tensor")
    T, K = shape
    if expert_weights is None:
        return T, K, MF_DTYPE_FP32
    w = expert_weights
    code = _WEIGHT_DTYPES.get(w.dtype)
    if code is None or w.shape != shape or not w.is_contiguous():
        raise ValueError("expert_weights must be contiguous BF16, FP32 or packed int32 with the "
                         "index map's shape")
    return T, K, code


def moe_dispatch(x: torch.Tensor, expanded_idx: torch.Tensor, output: torch.Tensor, *,
                 expert_weights: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``output[expanded_idx[t, j]] = expert_weights[t, j] * x[t]`` (in FP32, rounded
    once; a copy without weights).

    x: BF16 or FP32 [num_tokens, hidden]; output: BF16 or FP32 [rows, hidden]; unit
    last-dim strides, row strides multiples of 8, hidden a multiple of 8.  expanded_idx:
    int32 [num_tokens, top_k]; an entry outside the rows moves nothing, and no row may be
    named twice.  expert_weights: BF16, FP32 or packed int32 routing words.  Rows that no
    entry names are left as they were.  Returns ``output``.
    """
    x_rows, x_width, x_ld, x_dtype = _matrix(x, "x")
    rows, hidden, out_ld, out_dtype = _matrix(output, "output", written=True)
    T, K, wdt = _slots(expanded_idx, expert_weights)
    _req(x_rows == T and x_width == hidden,
         "x, output and the map disagree on num_tokens or hidden")
    _int32(hidden | K)
    dev = output.device
    _same_device(dev, x, expanded_idx, expert_weights)
    st = _on_device(dev, lib().moe_dispatch, x.data_ptr(), x_dtype, x_ld, _ptr(expert_weights),
                    wdt, expanded_idx.data_ptr(), output.data_ptr(), out_dtype, rows, out_ld, T,
                    hidden, K, _stream_ptr(stream, dev))
    check(st, "moe_dispatch")
    return output


def moe_combine(permuted: torch.Tensor, expert_weights: torch.Tensor, expanded_idx: torch.Tensor,
                output: torch.Tensor, *,
                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``output[t] = sum over j of expert_weights[t, j] * permuted[expanded_idx[t, j]]``,
    in FP32 in ascending j, rounded once: the finalize without its norm.

    permuted: BF16 or FP32 [rows, >= hidden]; output: BF16 or FP32 [num_tokens, hidden];
    unit last-dim strides, row strides multiples of 8, hidden a multiple of 8.
    expert_weights: BF16, FP32 or packed int32 routing words [num_tokens, top_k];
    expanded_idx: int32 of the same shape; an entry outside the rows contributes zero.
    Returns ``output``.
    """
    rows, width, ld, dtype = _matrix(permuted, "permuted")
    out_rows, hidden, out_ld, out_dtype = _matrix(output, "output", written=True)
    _req(expert_weights is not None, "expert_weights are required (moe_permuted_row_sum has none)")
    T, K, wdt = _slots(expanded_idx, expert_weights)
    _req(out_rows == T, "output and the map disagree on num_tokens")
    _req(width >= hidden, "permuted has fewer columns than output")
    _int32(hidden | K)
    dev = output.device
    _same_device(dev, permuted, expert_weights, expanded_idx)
    st = _on_device(dev, lib().moe_combine, permuted.data_ptr(), dtype, rows, ld,
                    expert_weights.data_ptr(), wdt, expanded_idx.data_ptr(), output.data_ptr(),
                    out_dtype, out_ld, T, hidden, K, _stream_ptr(stream, dev))
    check(st, "moe_combine")
    return output


def moe_combine_backward(grad_output: torch.Tensor, permuted: torch.Tensor | None,
                         expert_weights: torch.Tensor | None, expanded_idx: torch.Tensor,
                         grad_permuted: torch.Tensor | None, grad_weights: torch.Tensor | None, *,
                         stream: torch.cuda.Stream | None = None
                         ) -> tuple[torch.Tensor | None, torch.Tensor | None]:
    """Gradients of ``moe_combine``, in one pass over the rows::

        grad_permuted[expanded_idx[t, j]] = expert_weights[t, j] * grad_output[t]
        grad_weights[t, j] = dot(permuted[expanded_idx[t, j]], grad_output[t])

    Either may be None (not wanted); permuted may then be None without grad_weights, and
    expert_weights without grad_permuted.  grad_output: BF16 or FP32 [num_tokens, hidden];
    permuted: BF16 or FP32 [rows, hidden]; grad_permuted: the same shape and dtype;
    grad_weights: contiguous BF16 or FP32 [num_tokens, top_k], 0 for an entry outside the
    rows.  Rows that no entry names are left as they were; where grad_permuted is wanted no
    row may be named twice.  Returns ``(grad_permuted, grad_weights)``.
    """
    go_rows, hidden, go_ld, go_dtype = _matrix(grad_output, "grad_output")
    _req(grad_permuted is not None or grad_weights is not None, "no gradient is wanted")
    _req(grad_weights is None or permuted is not None, "grad_weights needs permuted")
    _req(grad_permuted is None or expert_weights is not None, "grad_permuted needs expert_weights")
    T, K, wdt = _slots(expanded_idx, expert_weights)
    _req(go_rows == T, "grad_output and the map disagree on num_tokens")
    like = permuted if permuted is not None else grad_permuted
    rows, width, ld, dtype = _matrix(like, "permuted")
    _req(width == hidden, "shapes disagree on hidden")
    gp_ld = hidden
    if grad_permuted is not None:
        gp_rows, gp_width, gp_ld, gp_dtype = _matrix(grad_permuted, "grad_permuted", written=True)
        _req(gp_rows == rows and gp_width == width and gp_dtype == dtype,
             "grad_permuted must have permuted's shape and dtype")
    gw_dtype = MF_DTYPE_FP32
    if grad_weights is not None:
        _req(grad_weights.dtype in _VALUE_DTYPES and grad_weights.shape == (T, K) and
             grad_weights.is_contiguous(),
             "grad_weights must be contiguous BF16 or FP32 with the index map's shape")
        gw_dtype = _VALUE_DTYPES[grad_weights.dtype]
    _int32(hidden | K)
    dev = grad_output.device
    _same_device(dev, permuted, expert_weights, expanded_idx, grad_permuted, grad_weights)
    st = _on_device(dev, lib().moe_combine_backward, grad_output.data_ptr(), go_dtype, go_ld,
                    _ptr(permuted), dtype, rows, ld, _ptr(expert_weights), wdt,
                    expanded_idx.data_ptr(), _ptr(grad_permuted), gp_ld, _ptr(grad_weights),
                    gw_dtype, T, hidden, K, _stream_ptr(stream, dev))
    check(st, "moe_combine_backward")
    return grad_permuted, grad_weights
