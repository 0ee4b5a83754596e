"""Refusals of the 4-bit floating point entry points (CPU only: fake pointers that are
never dereferenced, tensors without storage), and the tests' own reference."""
import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf
from moe_finalize_rmsnorm_gb300 import _abi
from moe_finalize_rmsnorm_gb300.build import build

import fp4_common as fp4

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, CUDA, TIMEOUT, INVALID = range(9)
BIG = 2 ** 31
# buffers far apart
A, B, C, D, E, F, G, H = (0x100000000 * i for i in range(1, 9))
MX, NV, U8, I32, F32 = fp4.MX, fp4.NV, torch.uint8, torch.int32, torch.float32


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


def quantize(lib, x=A, xdt=0, xs=64, f=B, q=C, qs=32, s=D, ss=16, fmt=0, rows=4, k=64):
    return lib.moe_quantize_fp4(x, xdt, xs, f, q, qs, s, ss, fmt, rows, k, None)


def dequantize(lib, q=A, qs=32, s=B, ss=16, fmt=0, out=C, odt=0, os=64, rows=4, k=64):
    return lib.moe_dequantize_fp4(q, qs, s, ss, fmt, out, odt, os, rows, k, None)


def gemm(lib, x=A, xr=10, xs=32, sc=B, scs=16, ri=C, w=D, ws=32, we=32 * 32, wsc=E, wscs=16,
         wsce=16 * 32, fmt=0, f=F, off=G, out=H, odt=0, os=32, rows=10, E_=4, n=32, k=64):
    return lib.moe_grouped_gemm_fp4(x, xr, xs, sc, scs, ri, w, ws, we, wsc, wscs, wsce, fmt, f, off,
                                    out, odt, os, rows, E_, n, k, None)


def test_sizes(lib):
    for call in (quantize, dequantize, gemm):
        for k in (0, 16, 48, 2 ** 20 + 32, -32):
            assert call(lib, k=k) == UNSUP, (call, k)
        for fmt in (-1, 2):
            assert call(lib, fmt=fmt) == INVALID
        for rows in (-1, BIG):
            assert call(lib, rows=rows) == SHAPE
    for n in (0, 4, 12, 2 ** 20 + 8):
        assert gemm(lib, n=n) == UNSUP
    for e in (0, 1025):
        assert gemm(lib, E_=e) == UNSUP


def test_strides(lib):
    for bad in (0, 16, 40, -32, 2 ** 36):
        assert quantize(lib, qs=bad) == SHAPE and dequantize(lib, qs=bad) == SHAPE, bad
        assert gemm(lib, xs=bad) == SHAPE and gemm(lib, ws=bad) == SHAPE, bad
    for bad in (0, 8, 24, -16, 2 ** 31, 2 ** 36):
        assert quantize(lib, ss=bad) == SHAPE and dequantize(lib, ss=bad) == SHAPE, bad
        assert gemm(lib, scs=bad) == SHAPE and gemm(lib, wscs=bad) == SHAPE, bad
    for bad in (56, 68, 0):
        assert quantize(lib, xs=bad) == SHAPE and dequantize(lib, os=bad) == SHAPE
    assert gemm(lib, os=24) == SHAPE and gemm(lib, os=36) == SHAPE
    # an expert inside the one before
    assert gemm(lib, we=32 * 31) == SHAPE and gemm(lib, wsce=16 * 30) == SHAPE
    assert gemm(lib, we=32 * 32 + 8) == SHAPE and gemm(lib, wsce=16 * 32 + 8) == SHAPE
    # scales of blocks of 16 need wider rows
    assert quantize(lib, k=512, xs=512, qs=256, ss=16) != SHAPE
    assert quantize(lib, k=512, xs=512, qs=256, ss=16, fmt=1) == SHAPE
    assert gemm(lib, xr=9, ri=None) == SHAPE and gemm(lib, xr=0) == SHAPE


def test_dtypes_null_and_alignment(lib):
    assert quantize(lib, xdt=2) == DTYPE and dequantize(lib, odt=2) == DTYPE
    assert gemm(lib, odt=2) == DTYPE
    assert gemm(lib, off=None) == INVALID
    for call, names in ((quantize, dict(x=A, q=C, s=D)), (dequantize, dict(q=A, s=B, out=C)),
                        (gemm, dict(x=A, sc=B, w=D, wsc=E, out=H))):
        for name, at in names.items():
            assert call(lib, **{name: None}) == NULL, (call, name)
            assert call(lib, **{name: at + 8}) == ALIGN, (call, name)
    for name, at in (("ri", C), ("f", F), ("off", G)):
        assert gemm(lib, **{name: at + 2}) == ALIGN, name
    assert quantize(lib, f=B + 2) == ALIGN


def test_overlap(lib):
    assert quantize(lib, q=A) == ALIGN and quantize(lib, s=A + 2 * 4 * 64 - 16) == ALIGN
    assert quantize(lib, s=C + 32 * 3 + 16) == ALIGN and quantize(lib, f=C + 16) == ALIGN
    assert quantize(lib, f=D + 16 * 3) == ALIGN
    assert dequantize(lib, out=A + 32 * 3) == ALIGN and dequantize(lib, out=B + 48) == ALIGN


def test_nothing_to_do(lib):
    assert quantize(lib, rows=0, x=None, q=None, s=None) == OK
    assert dequantize(lib, rows=0, q=None, s=None, out=None) == OK
    assert gemm(lib, rows=0, x=None, out=None) == OK


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def pair(*shape, k=64, fmt=MX):
    return mf.moe_fp4_empty(shape, k, fmt, device="meta")


def off(E):
    return meta(E + 1, dtype=I32)


@pytest.mark.parametrize("call", [
    lambda: mf.moe_fp4_empty((4,), 48, MX),
    lambda: mf.moe_fp4_empty((4,), 64, torch.float32),
    lambda: mf.moe_quantize_fp4(meta(4, 64, dtype=torch.float16), *pair(4)),
    lambda: mf.moe_quantize_fp4(meta(5, 64), *pair(4)),
    lambda: mf.moe_quantize_fp4(meta(4, 72), *pair(4)),
    lambda: mf.moe_quantize_fp4(meta(4, 64), *pair(2, 2)),
    lambda: mf.moe_quantize_fp4(meta(4, 64), pair(4)[0], pair(4, fmt=NV)[1][:, :2]),
    lambda: mf.moe_quantize_fp4(meta(4, 64), pair(4)[0], pair(4)[1].view(U8)),
    lambda: mf.moe_quantize_fp4(meta(4, 64), pair(4)[0].view(torch.int8), pair(4)[1]),
    lambda: mf.moe_quantize_fp4(meta(4, 64), pair(1)[0].expand(4, 32), pair(4)[1]),
    lambda: mf.moe_quantize_fp4(meta(4, 64), *pair(4), factor=meta(2, dtype=F32)),
    lambda: mf.moe_quantize_fp4(meta(4, 64), *pair(4), factor=meta(1)),
    lambda: mf.moe_dequantize_fp4(*pair(4), meta(4, 96)),
    lambda: mf.moe_dequantize_fp4(*pair(4), meta(4, 64, dtype=torch.float16)),
    lambda: mf.moe_dequantize_fp4(*pair(4), meta(1, 64).expand(4, 64)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(2, 32, fmt=NV), off(2), meta(6, 32)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(2, 32, k=96), off(2), meta(6, 32)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(2, 32), off(3), meta(6, 32)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(2, 32), None, meta(6, 32)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(5), *pair(2, 32), off(2), meta(6, 32)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(2, 32), off(2), meta(6, 40)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(32), off(2), meta(6, 32)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(2, 32), off(2), meta(6, 32),
                                    factor=meta(3, dtype=F32)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(2, 32), off(2), meta(6, 32),
                                    row_index=meta(5, dtype=I32)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(0), *pair(2, 32), off(2), meta(6, 32),
                                    row_index=meta(6, dtype=I32)),
    # a last row of scales at the end of its memory
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), pair(1, 1)[0], meta(1, 1, 2, dtype=U8).view(MX),
                                    off(1), meta(6, 1)),
    lambda: mf.moe_grouped_gemm_fp4(pair(1)[0], meta(1, 2, dtype=U8).view(MX), *pair(1, 32), off(1),
                                    meta(1, 32)),
    # right but for the device
    lambda: mf.moe_quantize_fp4(meta(4, 64), *pair(4)),
    lambda: mf.moe_dequantize_fp4(*pair(4), meta(4, 64)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(2, 32), off(2), meta(6, 32)),
    # sizes that the C interface's 32 bits do not hold
    lambda: mf.moe_quantize_fp4(meta(1, 2 ** 32 + 64), *pair(1, k=2 ** 32 + 64)),
    lambda: mf.moe_grouped_gemm_fp4(*pair(6), *pair(1, 2 ** 32 + 32), off(1),
                                    meta(6, 2 ** 32 + 32)),
])
def test_binding_refuses(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("k", [32, 96, 2880, 4096])
def test_allocation(fmt, k):
    q, s = mf.moe_fp4_empty((3, 5), k, fmt, device="cpu")
    assert q.shape == (3, 5, k // 2) and s.shape == (3, 5, k // fp4.BLOCK[fmt])
    assert s.dtype == fmt and s.stride(1) % 16 == 0 and s.data_ptr() % 16 == 0


def test_reference_scales():
    """The reference's scales against torch's own conversions."""
    b = torch.arange(256, dtype=torch.uint8)
    assert torch.equal(fp4.scale_values(b.view(MX)).nan_to_num(-1.0),
                       b.view(MX).double().nan_to_num(-1.0))
    assert torch.equal(fp4.scale_values(b[:128].view(NV)).nan_to_num(-1.0),
                       b[:128].view(NV).double().nan_to_num(-1.0))
    x = torch.randn((200, 64), dtype=torch.float64).mul(100).float()
    _, byte = fp4.quantize(x, NV)
    want = (x.double().view(200, 4, 16).abs().amax(-1) / 6).float().to(NV).view(U8)
    assert torch.equal(byte, want)
    _, byte = fp4.quantize(x, MX)
    want = torch.frexp(x.view(200, 2, 32).abs().amax(-1)).exponent - 3 + 127
    assert torch.equal(byte.int(), want.int())


def test_reference_values_are_nearest():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((50, 96), generator=g)
    for fmt in (MX, NV):
        codes, byte = fp4.quantize(x, fmt)
        s = byte.view(fmt)
        v = fp4.values(fp4.pack(codes), s)
        grid = torch.cat((fp4.MAGNITUDES, -fp4.MAGNITUDES))
        scale = fp4.scale_values(s).repeat_interleave(fp4.BLOCK[fmt], dim=-1)
        best = (x.double().unsqueeze(-1) - grid * scale.unsqueeze(-1)).abs().amin(-1)
        assert torch.equal((x.double() - v).abs(), best)
