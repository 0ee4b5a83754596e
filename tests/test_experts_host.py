"""Refusals of the expert-layer entry points (CPU only: nothing here reaches a
kernel; the C calls get fake pointers that are never dereferenced)."""
import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf
from moe_finalize_rmsnorm_gb300 import _abi
from moe_finalize_rmsnorm_gb300.build import build

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, CUDA, TIMEOUT, INVALID = range(9)
A, MIS, ODD = 0x10000, 0x10008, 0x10002
BIG = 2 ** 31


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


def permutation(lib, ids=A, packed=0, T=4, K=8, E=16, off=A, idx=A, tok=A):
    return lib.moe_expert_permutation(ids, packed, T, K, E, off, idx, tok, None)


def test_permutation_refusals(lib):
    for kw in (dict(E=0), dict(E=1025), dict(K=0), dict(K=33)):
        assert permutation(lib, **kw) == UNSUP, kw
    assert permutation(lib, T=-1) == SHAPE
    assert permutation(lib, T=BIG // 8, K=8) == SHAPE
    for name in ("ids", "off", "idx", "tok"):
        assert permutation(lib, **{name: None}) == NULL, name
    for name in ("ids", "idx", "tok"):
        assert permutation(lib, **{name: MIS}) == ALIGN, name
    assert permutation(lib, off=ODD) == ALIGN
    assert permutation(lib, T=0, ids=None, idx=None, tok=None, off=None) == NULL


def row_sum(lib, p=A, pdt=0, rows=10, ld=64, idx=A, out=A, odt=0, T=4, H=64, K=2):
    return lib.moe_permuted_row_sum(p, pdt, rows, ld, idx, out, odt, T, H, K, None)


def test_row_sum_refusals(lib):
    for kw in (dict(H=0), dict(H=4), dict(H=12), dict(H=2 ** 20 + 8), dict(K=0), dict(K=33)):
        assert row_sum(lib, **kw) == UNSUP, kw
    for kw in (dict(rows=-1), dict(T=-1), dict(ld=56), dict(ld=68), dict(T=BIG)):
        assert row_sum(lib, **kw) == SHAPE, kw
    assert row_sum(lib, pdt=2) == DTYPE and row_sum(lib, odt=2) == DTYPE
    for name in ("p", "idx", "out"):
        assert row_sum(lib, **{name: None}) == NULL, name
    assert row_sum(lib, p=MIS) == ALIGN and row_sum(lib, out=MIS) == ALIGN
    assert row_sum(lib, idx=ODD) == ALIGN
    assert row_sum(lib, T=0, p=None, idx=None, out=None) == OK


def gemm(lib, x=A, xr=10, xs=64, ri=None, w=A, ws=64, we=64 * 32, off=A, out=A, odt=0, os=32,
         rows=10, E=4, n=32, k=64):
    return lib.moe_grouped_gemm(x, xr, xs, ri, w, ws, we, off, out, odt, os, rows, E, n, k, None)


def dgrad(lib, dy=A, ds=32, w=A, ws=64, we=64 * 32, off=A, dx=A, odt=0, os=64, rows=10, E=4, n=32,
          k=64):
    return lib.moe_grouped_gemm_dgrad(dy, ds, w, ws, we, off, dx, odt, os, rows, E, n, k, None)


def wgrad(lib, dy=A, ds=32, x=A, xr=10, xs=64, ri=None, off=A, dw=A, odt=0, acc=0, rows=10, E=4,
          n=32, k=64):
    return lib.moe_grouped_gemm_wgrad(dy, ds, x, xr, xs, ri, off, dw, odt, acc, rows, E, n, k, None)


def test_grouped_gemm_refusals(lib):
    for call in (gemm, dgrad, wgrad):
        for kw in (dict(E=0), dict(E=1025), dict(n=0), dict(n=36), dict(k=0), dict(k=60),
                   dict(n=2 ** 20 + 8), dict(k=2 ** 20 + 8)):
            assert call(lib, **kw) == UNSUP, (call, kw)
        assert call(lib, rows=-1) == SHAPE
        assert call(lib, rows=BIG) == SHAPE
        for odt in (2, 5):
            assert call(lib, odt=odt) == DTYPE, call
        assert call(lib, off=ODD) == ALIGN
        assert call(lib, off=None) == NULL
    for kw in (dict(xs=56), dict(xs=68), dict(ws=56), dict(ws=68), dict(os=24), dict(os=36),
               dict(we=64 * 32 - 8), dict(we=64 * 32 + 4), dict(we=-64 * 32), dict(xr=9),
               dict(xr=0, ri=A), dict(xr=-1), dict(xs=2 ** 36)):
        assert gemm(lib, **kw) == SHAPE, kw
    for kw in (dict(ds=24), dict(ds=36), dict(ws=56), dict(os=56), dict(we=0)):
        assert dgrad(lib, **kw) == SHAPE, kw
    for kw in (dict(ds=24), dict(xs=56), dict(xr=9), dict(xr=0, ri=A)):
        assert wgrad(lib, **kw) == SHAPE, kw
    for call, names in ((gemm, ("x", "w", "out")), (dgrad, ("dy", "w", "dx")),
                        (wgrad, ("dy", "x", "dw"))):
        for name in names:
            assert call(lib, **{name: None}) == NULL, (call, name)
            assert call(lib, **{name: MIS}) == ALIGN, (call, name)
    assert gemm(lib, ri=ODD) == ALIGN and wgrad(lib, ri=ODD) == ALIGN
    # zero rows: a no-op, whatever the pointers (the weights' gradient only when it accumulates)
    assert gemm(lib, rows=0, x=None, w=None, off=None, out=None) == OK
    assert dgrad(lib, rows=0, dy=None, w=None, off=None, dx=None) == OK
    assert wgrad(lib, rows=0, acc=1, dy=None, x=None, off=None) == OK
    assert wgrad(lib, rows=0, dw=None) == NULL


def gemv(lib, x=A, xr=10, xs=256, ri=None, w=A, sc=A, sdt=0, z=None, g=64, off=A, out=A, odt=0,
         os=33, rows=10, E=4, n=33, k=256):
    return lib.moe_grouped_gemv_int4(x, xr, xs, ri, w, sc, sdt, z, g, off, out, odt, os, rows, E, n,
                                     k, None)


def test_gemv_int4_refusals(lib):
    for kw in (dict(E=0), dict(E=1025), dict(n=0), dict(n=2 ** 20 + 1), dict(k=0), dict(k=16),
               dict(g=0), dict(g=16), dict(g=256), dict(g=-32), dict(g=128, k=192, xs=192),
               dict(k=2 ** 21, xs=2 ** 21)):
        assert gemv(lib, **kw) == UNSUP, kw
    for kw in (dict(rows=-1), dict(rows=BIG), dict(xr=9), dict(xr=0, ri=A), dict(xs=248),
               dict(xs=260), dict(os=32)):
        assert gemv(lib, **kw) == SHAPE, kw
    assert gemv(lib, sdt=2) == DTYPE and gemv(lib, odt=2) == DTYPE
    assert gemv(lib, off=None) == INVALID
    for name in ("x", "w", "sc", "out"):
        assert gemv(lib, **{name: None}) == NULL, name
    assert gemv(lib, x=MIS) == ALIGN and gemv(lib, w=MIS) == ALIGN
    for name in ("sc", "off", "out", "ri", "z"):
        assert gemv(lib, **{name: ODD}) == ALIGN, name
    assert gemv(lib, rows=0, x=None, w=None, sc=None, off=None, E=1, out=None) == OK


# ---------------------------------------------------------------------------
# the binding's own checks (CPU tensors: every call is refused)

def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def refused(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_binding_refuses_bad_metadata():
    u8 = torch.zeros((2, 16, 32), dtype=torch.uint8)
    x, w, off, out = bf(6, 64), bf(2, 16, 64), i32(3), bf(6, 16)
    refused("same CUDA device", mf.moe_grouped_gemm, x, w, off, out)  # all well formed, but on CPU
    refused("unit last-dim", mf.moe_grouped_gemm, x.float(), w, off, out)
    refused("unit last-dim", mf.moe_grouped_gemm, bf(64, 6).t(), w, off, out)
    refused("unit last-dim", mf.moe_grouped_gemm, x, w.transpose(1, 2), off, out)
    refused("weight", mf.moe_grouped_gemm, x, w[0], off, out)
    refused("expert_offsets", mf.moe_grouped_gemm, x, w, i32(2), out)
    refused("expert_offsets", mf.moe_grouped_gemm, x, w, off.long(), out)
    refused("expert_offsets", mf.moe_grouped_gemm, x, w, i32(6)[::2], out)
    refused("disagree", mf.moe_grouped_gemm, x, w, off, bf(6, 24))
    refused("disagree", mf.moe_grouped_gemm, bf(6, 72), w, off, out)
    refused("fewer rows", mf.moe_grouped_gemm, bf(5, 64), w, off, out)
    refused("row_index", mf.moe_grouped_gemm, x, w, off, out, row_index=i32(5))
    refused("needs rows", mf.moe_grouped_gemm, bf(0, 64), w, off, out, row_index=i32(6))
    refused("overlap", mf.moe_grouped_gemm, x, w, off, bf(1, 16).expand(6, 16))
    refused("unit last-dim", mf.moe_grouped_gemm, x, w, off, out.half())
    refused("disagree", mf.moe_grouped_gemm_dgrad, bf(6, 24), w, off, bf(6, 64))
    refused("disagree", mf.moe_grouped_gemm_dgrad, bf(5, 16), w, off, bf(6, 64))
    refused("same CUDA", mf.moe_grouped_gemm_dgrad, bf(6, 16), w, off, bf(6, 64))
    refused("grad_weight", mf.moe_grouped_gemm_wgrad, bf(6, 16), x, off, w.transpose(1, 2))
    refused("grad_weight", mf.moe_grouped_gemm_wgrad, bf(6, 16), x, off, w.half())
    refused("fewer rows", mf.moe_grouped_gemm_wgrad, bf(6, 16), bf(5, 64), off, w)
    refused("same CUDA", mf.moe_grouped_gemm_wgrad, bf(6, 16), x, off, w)
    sc = bf(2, 16, 2)
    refused("same CUDA", mf.moe_grouped_gemv_int4, x, u8, sc, off, out)
    refused("uint8", mf.moe_grouped_gemv_int4, x, u8.int(), sc, off, out)
    refused("scales", mf.moe_grouped_gemv_int4, x, u8, sc[:, :8], off, out)
    refused("groups", mf.moe_grouped_gemv_int4, x, u8, bf(2, 16, 4), off, out)
    refused("groups", mf.moe_grouped_gemv_int4, x, u8, bf(2, 16, 0), off, out)
    refused("zeros", mf.moe_grouped_gemv_int4, x, u8, sc, off, out, zeros=u8[:, :, :1])
    refused("one expert", mf.moe_grouped_gemv_int4, x, u8, sc, None, out)
    refused("2-D int32", mf.moe_expert_permutation, i32(8), 4)
    refused("2-D int32", mf.moe_expert_permutation, i32(8, 2).long(), 4)
    refused("same CUDA", mf.moe_expert_permutation, i32(8, 2), 4)
    refused("disagree|columns", mf.moe_permuted_row_sum, bf(6, 16), i32(3, 2), bf(3, 24))
    refused("expanded_idx", mf.moe_permuted_row_sum, bf(6, 16), i32(4, 2), bf(3, 16))
    refused("same CUDA", mf.moe_permuted_row_sum, bf(6, 16), i32(3, 2), bf(3, 16))
