"""Accuracy of the expert layer's sums, against float64, with bounds that follow from the
order in which each kernel adds.

`within` counts errors in steps of 2^-23 of the terms' magnitudes.  A tensor-core
accumulator takes the sum of 16 products at a time and truncates: at most 2^-22 of the
running magnitude (two bits) each time, so C summed values in one accumulator lose
C / 16 * 2^-22.  Sums that leave the tensor cores every 640 values lose 40 * 2^-22, and
each addition outside 2^-24.
"""
import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf
from tests.test_experts_gpu import BF16, FP32, offsets_of, randn, within

pytestmark = pytest.mark.gpu


def one_accumulator(summed):
    return 2 * (summed / 16 + 1)


def moved_sums(summed):
    return 2 * (40 + summed / 640 + 1)


def positive(shape, seed):
    """Values of one sign: every truncated bit counts in the same direction."""
    return randn(shape, seed, FP32).abs().to(BF16)


# 32768 values are the most that one accumulator takes for a BF16 result
LONG = [4096, 32768, 32776, 600000]


@pytest.mark.parametrize("k", [*LONG, 2 ** 20])
def test_bf16_results_of_long_sums(cuda_lib, k):
    """Forward and the rows' gradient; 72 rows are too many for the few-rows kernel."""
    rows, n = 72, 16
    x, w = positive((rows, k), 1), positive((1, n, k), 2)
    off = offsets_of([rows])
    index = torch.arange(rows, dtype=torch.int32, device="cuda")
    ref = x.double() @ w[0].double().t()
    dy, wt = x, w.transpose(1, 2).contiguous()          # [1, k, n]: sums over k again
    terms = one_accumulator(k) if k <= 32768 else moved_sums(k)
    for call in (lambda o: mf.moe_grouped_gemm(x, w, off, o),
                 lambda o: mf.moe_grouped_gemm(x, w, off, o, row_index=index),
                 lambda o: mf.moe_grouped_gemm_dgrad(dy, wt, off, o)):
        out = torch.empty((rows, n), dtype=BF16, device="cuda")
        exact = torch.empty((rows, n), dtype=FP32, device="cuda")
        call(out)
        call(exact)
        within(exact, ref, ref, moved_sums(k), FP32)
        within(out, ref, ref, terms, BF16)
        if k > 32768:           # the same sums, rounded once
            assert torch.equal(out, exact.to(BF16))


@pytest.mark.parametrize("many", LONG)
@pytest.mark.parametrize("gather", [False, True])
def test_bf16_weight_gradients_of_long_sums(cuda_lib, many, gather):
    """Added to minus the rounded result, so that the sum's own error shows; experts with
    short sums, and none, before and behind it."""
    n, k = 136, 264
    sizes = [70, 0, many, 33, 0]
    rows = sum(sizes) + 3
    dy, x = positive((rows, n), 1), positive((rows, k), 2)
    index = torch.arange(rows, dtype=torch.int32, device="cuda") if gather else None
    off = offsets_of(sizes)
    ref = torch.stack([a.t() @ b for a, b in zip(dy[:-3].double().split(sizes),
                                                x[:-3].double().split(sizes))])
    base = -ref.to(BF16)
    out = base.clone()
    mf.moe_grouped_gemm_wgrad(dy, x, off, out, row_index=index, accumulate=True)
    lo = 0
    for e, m in enumerate(sizes):
        terms = (one_accumulator(m) if m <= 32768 else moved_sums(m)) + 1
        within(out[e], ref[e] + base[e].double(), ref[e], terms, BF16)
        lo += m
    assert torch.equal(out[1], base[1]) and torch.equal(out[4], base[4])
    written = torch.full((len(sizes), n, k), 7.0, dtype=BF16, device="cuda")
    exact = torch.empty((len(sizes), n, k), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm_wgrad(dy, x, off, written, row_index=index)
    mf.moe_grouped_gemm_wgrad(dy, x, off, exact, row_index=index)
    for e, m in enumerate(sizes):
        terms = one_accumulator(m) if m <= 32768 else moved_sums(m)
        within(written[e], ref[e], ref[e], terms, BF16)
        within(exact[e], ref[e], ref[e], moved_sums(m), FP32)
    if many > 32768:
        assert torch.equal(written[2], exact[2].to(BF16))


@pytest.mark.parametrize("rows,experts,n,k", [(1, 1, 264, 7168), (8, 8, 512, 4096),
                                              (64, 3, 136, 4104), (200, 100, 64, 1000),
                                              (33, 2, 40, 40)])
def test_few_rows_are_summed_in_short_pieces(cuda_lib, rows, experts, n, k):
    """64 values at a time (four products of 16), each stage's sum and the up to twelve
    warps' shares added in FP32."""
    sizes = [rows // experts + (e < rows % experts) for e in range(experts)]
    off = offsets_of(sizes)
    x, w = positive((rows, k), 1), positive((experts, n, k), 2)
    out = torch.empty((rows, n), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm(x, w, off, out)
    ref = torch.cat([r @ m.t() for r, m in zip(x.double().split(sizes), w.double())])
    stages = -(-k // 64)
    within(out, ref, ref, 2 * 4 + (stages + 12) / 2, FP32)
    # the truncation of a piece is at most 4 * 2^-22, on average half; what the sums of the
    # stages round off cancels
    assert (out.double() - ref).norm() < 5e-7 * ref.norm()
