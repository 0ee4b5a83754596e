"""Refusals of moe_dispatch, moe_combine and moe_combine_backward (CPU only: fake
pointers that are never dereferenced, tensors without storage)."""
import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf
from moe_finalize_rmsnorm_gb300 import _abi
from moe_finalize_rmsnorm_gb300.build import build

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, CUDA, TIMEOUT, INVALID = range(9)
BIG = 2 ** 31
# buffers far apart
A, B, C, D, E, F = (0x100000000 * i for i in range(1, 7))


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


def dispatch(lib, x=A, xdt=0, xs=64, w=B, wdt=1, idx=C, out=D, odt=0, rows=10, os=64, T=4, H=64,
             K=2):
    return lib.moe_dispatch(x, xdt, xs, w, wdt, idx, out, odt, rows, os, T, H, K, None)


def combine(lib, p=A, pdt=0, rows=10, ps=64, w=B, wdt=1, idx=C, out=D, odt=0, os=64, T=4, H=64,
            K=2):
    return lib.moe_combine(p, pdt, rows, ps, w, wdt, idx, out, odt, os, T, H, K, None)


def backward(lib, go=A, gdt=0, gs=64, p=B, pdt=0, rows=10, ps=64, w=C, wdt=1, idx=D, gp=E, gps=64,
             gw=F, gwdt=1, T=4, H=64, K=2):
    return lib.moe_combine_backward(go, gdt, gs, p, pdt, rows, ps, w, wdt, idx, gp, gps, gw, gwdt,
                                    T, H, K, None)


@pytest.mark.parametrize("call", [dispatch, combine, backward])
def test_sizes_and_strides(lib, call):
    for kw in (dict(H=0), dict(H=4), dict(H=12), dict(H=2 ** 20 + 8), dict(K=0), dict(K=33)):
        assert call(lib, **kw) == UNSUP, kw
    for kw in (dict(rows=-1), dict(rows=BIG), dict(T=-1), dict(T=BIG), dict(T=BIG // 2)):
        assert call(lib, **kw) == SHAPE, kw
    strides = dict(dispatch=("xs", "os"), combine=("ps", "os"), backward=("gs", "ps", "gps"))
    for name in strides[call.__name__]:
        for bad in (0, 56, 68, -64, 2 ** 36):
            assert call(lib, **{name: bad}) == SHAPE, (name, bad)


def test_dtypes(lib):
    assert dispatch(lib, xdt=2) == DTYPE and dispatch(lib, odt=2) == DTYPE
    assert dispatch(lib, wdt=3) == DTYPE
    assert combine(lib, pdt=2) == DTYPE and combine(lib, odt=2) == DTYPE
    assert combine(lib, wdt=3) == DTYPE
    for kw in (dict(gdt=2), dict(pdt=2), dict(wdt=3), dict(gwdt=2)):
        assert backward(lib, **kw) == DTYPE, kw


def test_null_and_alignment(lib):
    for name in ("x", "idx", "out"):
        assert dispatch(lib, **{name: None}) == NULL, name
    for name in ("p", "w", "idx", "out"):
        assert combine(lib, **{name: None}) == NULL, name
    for name in ("go", "p", "w", "idx"):
        assert backward(lib, **{name: None}) == NULL, name
    assert backward(lib, gp=None, gw=None) == INVALID
    for call, at in ((dispatch, dict(x=A, out=D)), (combine, dict(p=A, out=D)),
                     (backward, dict(go=A, p=B, gp=E))):
        for name, base in at.items():
            assert call(lib, **{name: base + 8}) == ALIGN, (call, name)
        assert call(lib, idx=dict(dispatch=C, combine=C, backward=D)[call.__name__] + 2) == ALIGN
    for call, w in ((dispatch, B), (combine, B), (backward, C)):
        assert call(lib, w=w + 2) == ALIGN                 # FP32 words
        assert call(lib, w=w + 1, wdt=0) == ALIGN          # BF16
    assert backward(lib, gw=F + 2) == ALIGN and backward(lib, gw=F + 1, gwdt=0) == ALIGN


def test_outputs_over_inputs(lib):
    x_bytes, rows_bytes, slots = 2 * 4 * 64, 2 * 10 * 64, 4 * 8
    for shift in (0, 16, x_bytes - 16, 16 - rows_bytes):
        assert dispatch(lib, out=A + shift) == ALIGN, shift
    for shift in (0, 16, rows_bytes - 16, 16 - x_bytes):
        assert combine(lib, out=A + shift) == ALIGN, shift
    for at in (B, C):
        assert dispatch(lib, out=at + slots - 16) == ALIGN
        assert combine(lib, out=at + slots - 16) == ALIGN
    for at, size in ((A, x_bytes), (B, rows_bytes), (C, slots), (D, slots)):
        assert backward(lib, gp=at + size - 16) == ALIGN, at
        assert backward(lib, gw=at + size - 4) == ALIGN, at
    assert backward(lib, gw=E + rows_bytes - 4) == ALIGN


def test_nothing_to_do(lib):
    assert dispatch(lib, T=0, x=None, idx=None, w=None) == OK
    assert dispatch(lib, rows=0, out=None) == OK
    assert combine(lib, T=0, w=None, idx=None, out=None) == OK
    assert backward(lib, T=0, go=None, p=None, w=None, idx=None) == OK
    assert backward(lib, rows=0, gw=None, p=None) == OK


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


I32, F32 = torch.int32, torch.float32


@pytest.mark.parametrize("call", [
    lambda: mf.moe_dispatch(meta(4, 64), meta(4, 2, dtype=torch.int64), meta(8, 64)),
    lambda: mf.moe_dispatch(meta(3, 64), meta(4, 2, dtype=I32), meta(8, 64)),
    lambda: mf.moe_dispatch(meta(4, 72), meta(4, 2, dtype=I32), meta(8, 64)),
    lambda: mf.moe_dispatch(meta(4, 64, dtype=torch.float16), meta(4, 2, dtype=I32), meta(8, 64)),
    lambda: mf.moe_dispatch(meta(4, 128)[:, ::2], meta(4, 2, dtype=I32), meta(8, 64)),
    lambda: mf.moe_dispatch(meta(4, 64), meta(4, 2, dtype=I32), meta(1, 64).expand(8, 64)),
    lambda: mf.moe_dispatch(meta(4, 64), meta(4, 2, dtype=I32), meta(8, 64),
                            expert_weights=meta(4, 3, dtype=F32)),
    lambda: mf.moe_dispatch(meta(4, 64), meta(4, 2, dtype=I32), meta(8, 64),
                            expert_weights=meta(2, 4, dtype=F32).t()),
    lambda: mf.moe_combine(meta(8, 64), None, meta(4, 2, dtype=I32), meta(4, 64)),
    lambda: mf.moe_combine(meta(8, 56), meta(4, 2), meta(4, 2, dtype=I32), meta(4, 64)),
    lambda: mf.moe_combine(meta(8, 64), meta(4, 2), meta(4, 2, dtype=I32), meta(5, 64)),
    lambda: mf.moe_combine(meta(8, 64), meta(4, 2, dtype=torch.float16), meta(4, 2, dtype=I32),
                           meta(4, 64)),
    lambda: mf.moe_combine(meta(8, 64), meta(4, 2), meta(8, dtype=I32), meta(4, 64)),
    lambda: mf.moe_combine_backward(meta(4, 64), meta(8, 64), meta(4, 2), meta(4, 2, dtype=I32),
                                    None, None),
    lambda: mf.moe_combine_backward(meta(4, 64), None, meta(4, 2), meta(4, 2, dtype=I32),
                                    meta(8, 64), meta(4, 2)),
    lambda: mf.moe_combine_backward(meta(4, 64), meta(8, 64), None, meta(4, 2, dtype=I32),
                                    meta(8, 64), meta(4, 2)),
    lambda: mf.moe_combine_backward(meta(4, 64), meta(8, 64), meta(4, 2), meta(4, 2, dtype=I32),
                                    meta(8, 64, dtype=F32), meta(4, 2)),
    lambda: mf.moe_combine_backward(meta(4, 64), meta(8, 64), meta(4, 2), meta(4, 2, dtype=I32),
                                    meta(9, 64), meta(4, 2)),
    lambda: mf.moe_combine_backward(meta(4, 64), meta(8, 64), meta(4, 2), meta(4, 2, dtype=I32),
                                    meta(8, 64), meta(4, 3)),
    lambda: mf.moe_combine_backward(meta(5, 64), meta(8, 64), meta(4, 2), meta(4, 2, dtype=I32),
                                    meta(8, 64), meta(4, 2)),
    # right but for the device
    lambda: mf.moe_dispatch(meta(4, 64), meta(4, 2, dtype=I32), meta(8, 64)),
    lambda: mf.moe_combine(meta(8, 64), meta(4, 2), meta(4, 2, dtype=I32), meta(4, 64)),
    lambda: mf.moe_combine_backward(meta(4, 64), meta(8, 64), meta(4, 2), meta(4, 2, dtype=I32),
                                    meta(8, 64), meta(4, 2)),
    # sizes that the C interface's 32 bits do not hold
    lambda: mf.moe_dispatch(meta(4, 2 ** 32 + 64), meta(4, 2, dtype=I32), meta(8, 2 ** 32 + 64)),
    lambda: mf.moe_combine(meta(8, 2 ** 32 + 64), meta(4, 2), meta(4, 2, dtype=I32),
                           meta(4, 2 ** 32 + 64)),
    lambda: mf.moe_combine_backward(meta(1, 64), meta(8, 64), None, meta(1, 2 ** 32 + 2, dtype=I32),
                                    None, meta(1, 2 ** 32 + 2)),
])
def test_binding_refuses(call):
    with pytest.raises(ValueError):
        call()


def test_one_row_keeps_no_stride():
    """A single row's columns may end anywhere: the stride that the kernels get is a multiple
    of 8 that covers them."""
    from moe_finalize_rmsnorm_gb300.combine import _matrix
    for width, ld in ((64, 64), (60, 64), (1, 8), (68, 72)):
        whole = torch.empty((1, 100), dtype=torch.bfloat16)
        assert _matrix(whole[:, :width], "t") == (1, width, ld, 0)
        assert _matrix(torch.empty((1, width)).expand(1, width), "t", written=True)[2] == ld
