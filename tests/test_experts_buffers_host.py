"""Refusals of buffers that overlap or are not aligned, and of sizes that do not fit (CPU
only: fake pointers, never dereferenced)."""
import pytest

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
