"""Refusals of buffers that overlap or are not aligned, and of sizes that do not fit (CPU
only: fake pointers, never dereferenced)."""
import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf
from moe_finalize_rmsnorm_gb300 import _abi
from moe_finalize_rmsnorm_gb300.build import build

ALIGN = 3
IDS, IDX, TOK, OFF = 0x100000, 0x200000, 0x300000, 0x400000


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


def permutation(lib, T=1000, K=8, E=16, **at):
    p = dict(ids=IDS, idx=IDX, tok=TOK, off=OFF)
    p.update(at)
    return lib.moe_expert_permutation(p["ids"], 0, T, K, E, p["off"], p["idx"], p["tok"], None)


def test_permutation_refuses_buffers_that_overlap(lib):
    size = 4 * 1000 * 8
    for a, b in (("ids", "idx"), ("ids", "tok"), ("idx", "tok")):
        at = dict(ids=IDS, idx=IDX, tok=TOK)[a]
        for shift in (0, 16, size - 16, 16 - size):
            assert permutation(lib, **{b: at + shift}) == ALIGN, (a, b, shift)
    for name, at in (("ids", IDS), ("idx", IDX), ("tok", TOK)):
        for shift in (0, size - 4, -4 * 16):
            assert permutation(lib, off=at + shift) == ALIGN, (name, shift)


def test_permutation_refuses_what_is_no_word(lib):
    for name, at in (("ids", IDS), ("idx", IDX), ("tok", TOK), ("off", OFF)):
        assert permutation(lib, **{name: at + 2}) == ALIGN, name


def test_sizes_beyond_32_bits_are_refused():
    """They are not cut to their lower half (2^32 + 16 experts are not 16)."""
    wide = 2 ** 32 + 16

    def meta(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    off, x, i32 = meta(2, dtype=torch.int32), meta(6, 64), torch.int32
    calls = [
        lambda: mf.moe_expert_permutation(meta(4, 2, dtype=i32), wide),
        lambda: mf.moe_expert_permutation(meta(4, 2, dtype=i32), -wide),
        lambda: mf.moe_expert_permutation(meta(4, wide, dtype=i32), 16),
        lambda: mf.moe_permuted_row_sum(meta(6, wide), meta(3, 2, dtype=i32), meta(3, wide)),
        lambda: mf.moe_permuted_row_sum(x, meta(3, wide, dtype=i32), meta(3, 64)),
        lambda: mf.moe_grouped_gemm(x, meta(1, wide, 64), off, meta(6, wide)),
        lambda: mf.moe_grouped_gemm(meta(6, wide), meta(1, 64, wide), off, meta(6, 64)),
        lambda: mf.moe_grouped_gemm_dgrad(meta(6, wide), meta(1, wide, 64), off, x),
        lambda: mf.moe_grouped_gemm_wgrad(meta(6, wide), x, off, meta(1, wide, 64)),
        lambda: mf.moe_grouped_gemv_int4(x, meta(1, wide, 32, dtype=torch.uint8),
                                         meta(1, wide, 2), None, meta(6, wide)),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()
