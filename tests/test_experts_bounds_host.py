"""The bounds of the expert layer's GPU tests reject results that are wrong by little: a
few of the summed values left out, FP32 results or scales rounded to BF16 (CPU only: the
mistakes are made here, in the expected values)."""
import pytest
import torch

from tests.experts_bounds import check, few_rows, int4, moved_sums, one_accumulator
from tests.test_experts_gpu import BF16, FP32, F64


def operands(rows, n, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, k), generator=g).to(BF16).to(F64)
    w = (torch.randn((n, k), generator=g) * k ** -0.5).to(BF16).to(F64)
    return x, w


def rejects(wrong, ref, mag, terms, dtype):
    check(ref.to(dtype), ref, mag, terms, dtype)      # the right result passes
    with pytest.raises(AssertionError):
        check(wrong.to(dtype), ref, mag, terms, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("k", [1000, 4096, 7168, 16384, 32768, 65536])
def test_a_block_of_the_sum_left_out(k, dtype):
    """The last 16 values (a product of the tensor cores), 8 of them, and any one in the
    middle of short sums."""
    x, w = operands(24, 64, k)
    ref, mag = x @ w.t(), x.abs() @ w.abs().t()
    bounds = [moved_sums(k)] if dtype == FP32 or k > 32768 else [one_accumulator(k)]
    bounds.append(few_rows(k))
    for terms in bounds:
        for lo, hi in ((k - 16, k), (k - 8, k), (0, 32)):
            rejects(ref - x[:, lo:hi] @ w[:, lo:hi].t(), ref, mag, terms, dtype)


@pytest.mark.parametrize("k", [40, 1000, 4096, 16384, 65536])
def test_fp32_results_rounded_to_bf16(k):
    x, w = operands(24, 64, k)
    ref, mag = x @ w.t(), x.abs() @ w.abs().t()
    for terms in (moved_sums(k), few_rows(k)):
        rejects(ref.to(BF16), ref, mag, terms, FP32)


@pytest.mark.parametrize("rows", [1, 8])
@pytest.mark.parametrize("k,group", [(4096, 128), (7168, 64), (16384, 32), (2880, 32), (96, 32)])
def test_4_bit_products(k, group, rows):
    g = torch.Generator().manual_seed(k)
    x, _ = operands(rows, 1, k)
    q = torch.randint(-8, 8, (64, k), generator=g).to(F64)
    s = (torch.rand((64, k // group), generator=g) * 0.02 + 0.001).to(FP32)

    def product(scales, columns=slice(None)):
        w = q * scales.to(F64).repeat_interleave(group, 1)
        return x[:, columns] @ w[:, columns].t(), x[:, columns].abs() @ w[:, columns].abs().t()

    ref, mag = product(s)
    terms = int4(k, group)
    for dtype in (BF16, FP32):
        for columns in (slice(k - 32, k), slice(k - 16, k), slice(0, 16)):
            rejects(ref - product(s, columns)[0], ref, mag, terms, dtype)
    rejects(ref.to(BF16), ref, mag, terms, FP32)
    rejects(product(s.to(BF16))[0], ref, mag, terms, FP32)
