"""Accuracy of the expert layer's sums against float64, with bounds that follow from the
order in which each kernel adds (tests/experts_bounds.py)."""
import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf
from tests.experts_bounds import check, few_rows, int4, moved_sums, one_accumulator
from tests.test_experts_gpu import (BF16, FP32, gathered, gen, int4_weights, offsets_of, padded,
                                    randn, weights, within)

pytestmark = pytest.mark.gpu


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


# ---------------------------------------------------------------------------
# values of either sign, every operation and result type

def split_product(a, b, sizes):
    """a's rows by expert times b[e], and the magnitudes."""
    parts = [(r, m) for r, m in zip(a.split(sizes), b)]
    return (torch.cat([r @ m for r, m in parts]),
            torch.cat([r.abs() @ m.abs() for r, m in parts]))


def terms_of(summed, dtype):
    return moved_sums(summed) if dtype == FP32 or summed > 32768 else one_accumulator(summed)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,k", [(264, 4096), (136, 7168), (1000, 1000), (64, 65536)])
def test_products(cuda_lib, n, k, dtype):
    sizes = [300, 0, 211, 1]
    rows = sum(sizes)
    w, off = weights(4, n, k, 1, 8), offsets_of(sizes)
    x = padded(rows, k, 2, 8)
    some = padded(90, k, 3, 0)
    index = torch.randint(-1, 91, (rows,), generator=gen(4), dtype=torch.int32).cuda()
    for a, ix in ((x, None), (some, index)):
        out = torch.empty((rows, n), dtype=dtype, device="cuda")
        mf.moe_grouped_gemm(a, w, off, out, row_index=ix)
        ref, mag = split_product(gathered(a, ix, rows), w.double().transpose(1, 2), sizes)
        check(out, ref, mag, terms_of(k, dtype), dtype)
    # the gradient of the rows sums over the other dimension
    wt = weights(4, k, n, 5, 8)
    out = torch.empty((rows, n), dtype=dtype, device="cuda")
    mf.moe_grouped_gemm_dgrad(x, wt, off, out)
    check(out, *split_product(x.double(), wt.double(), sizes), terms_of(k, dtype), dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("sizes,n,k", [([8, 0, 30, 26], 264, 4096), ([1], 1000, 7168),
                                       ([2] * 60, 72, 1416), ([0, 64], 40, 65536)])
def test_products_of_few_rows(cuda_lib, sizes, n, k, dtype):
    rows, E = sum(sizes), len(sizes)
    w, x = weights(E, n, k, 1, 8), padded(rows, k, 2, 8)
    index = torch.randint(0, rows, (rows,), generator=gen(4), dtype=torch.int32).cuda()
    for ix in (None, index):
        out = torch.empty((rows, n), dtype=dtype, device="cuda")
        mf.moe_grouped_gemm(x, w, offsets_of(sizes), out, row_index=ix)
        ref, mag = split_product(gathered(x, ix, rows), w.double().transpose(1, 2), sizes)
        check(out, ref, mag, few_rows(k), dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes", [[700, 0, 1, 5000], [64, 65, 128, 16384], [40000, 3]])
def test_weight_gradients(cuda_lib, sizes, accumulate, dtype):
    rows, n, k = sum(sizes), 136, 264
    dy, x = padded(rows, n, 1, 8), padded(rows, k, 2, 0)
    index = torch.randint(0, rows, (rows,), generator=gen(4), dtype=torch.int32).cuda()
    for ix in (None, index):
        base = randn((len(sizes), n, k), 3, dtype)
        out = base.clone()
        mf.moe_grouped_gemm_wgrad(dy, x, offsets_of(sizes), out, row_index=ix,
                                  accumulate=accumulate)
        a = gathered(x, ix, rows)
        for e, (g, r) in enumerate(zip(dy.double().split(sizes), a.split(sizes))):
            ref, mag = g.t() @ r, g.abs().t() @ r.abs()
            if accumulate:
                ref, mag = ref + base[e].double(), mag + base[e].double().abs()
            check(out[e], ref, mag, terms_of(len(g), dtype) + 1, dtype)


@pytest.mark.parametrize("rows", [1, 5, 6, 16, 24, 25, 70])
@pytest.mark.parametrize("n,k,group", [(515, 4096, 128), (64, 16384, 32), (101, 7168, 64),
                                       (33, 2880, 32), (40, 1408, 128), (7, 96, 32)])
def test_4_bit_products(cuda_lib, rows, n, k, group):
    """One matrix and three, scales of either type, zeros or none."""
    for sizes, dtype, scale_dtype, zeros in (([rows], FP32, FP32, False), ([rows], BF16, BF16, True),
                                             ([rows, 0, 3], FP32, BF16, True),
                                             ([1, rows, 2], BF16, FP32, False)):
        q, s, z, w = int4_weights(len(sizes), n, k, group, scale_dtype, zeros, rows)
        x = padded(sum(sizes), k, 2, 8)
        out = torch.empty((sum(sizes), n), dtype=dtype, device="cuda")
        mf.moe_grouped_gemv_int4(x, q, s, offsets_of(sizes), out, zeros=z)
        check(out, *split_product(x.double(), w.transpose(1, 2), sizes), int4(k, group), dtype)


@pytest.mark.parametrize("programmatic", [True, False])
def test_long_weight_gradients_in_a_graph(cuda_lib, programmatic):
    """The two launches of a call with a long sum, captured behind the product that makes
    their operand, added to and replayed: the bits of the eager calls."""
    sizes, n, k = [33000, 0, 500], 136, 264
    rows, off = sum(sizes), offsets_of(sizes)
    w, x, dy = weights(3, n, k, 1), padded(rows, k, 2, 0), padded(rows, n, 3, 0)
    start = randn((3, n, k), 4)

    def step(grad, made):
        mf.moe_grouped_gemm(x, w, off, made)
        mf.moe_grouped_gemm_wgrad(made, x, off, grad, accumulate=True)
        mf.moe_grouped_gemm_wgrad(dy, x, off, grad, accumulate=True)

    mf.set_programmatic_launch(programmatic)
    try:
        want, made = start.clone(), torch.empty((rows, n), dtype=BF16, device="cuda")
        step(want, made)
        step(want, made)
        got, made = start.clone(), torch.empty((rows, n), dtype=BF16, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(got, made)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    finally:
        mf.set_programmatic_launch(True)
