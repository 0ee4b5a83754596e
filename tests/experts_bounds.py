"""Error bounds of the expert layer's sums, by the order in which each kernel adds.

They count steps of 2^-23 of the terms' magnitudes S.  A tensor-core accumulator takes the
sum of 16 products at a time and truncates two bits at most: 2^-22 of the running magnitude
each time.  FP32 additions and multiply-adds outside round: 2^-24 each.
"""
from tests.test_experts_gpu import FP32, within

# FP32 results as a whole, in the Euclidean norm.  The longest sum inside the tensor cores
# is 640 values, 40 truncations: each loses half a step (2^-24) of the running sum on
# average, which itself is 2/3 of the final one on average over a random walk.
NORM = 40 * 2.0 ** -24 * 2 / 3


def one_accumulator(summed):
    """BF16 results of up to 32768 values."""
    return 2 * (summed / 16 + 1)


def moved_sums(summed):
    """FP32 results, and longer sums: 640 values in the tensor cores, the rest outside."""
    return 2 * (40 + summed / 640 + 1)


def few_rows(summed):
    """Up to 64 rows, or two an expert: a stage of 64 values in the tensor cores, the
    stages and the shares of up to 12 warps outside."""
    return 2 * 4 + (summed / 64 + 13) / 2


def int4(summed, group):
    """A group in the tensor cores, then a multiply-add a group and up to 16 warps."""
    return 2 * group / 16 + (summed / group + 17) / 2


def check(got, ref, mag, terms, dtype):
    within(got, ref, mag, terms, dtype)
    if dtype == FP32:
        off = (got.double() - ref).norm() / ref.norm().clamp_min(1e-300)
        assert off < NORM, f"off by {off:.2e} of the result"
