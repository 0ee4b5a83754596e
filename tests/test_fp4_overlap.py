"""moe_grouped_gemm_fp4 refuses an output over its inputs (on the CPU: fake pointers that are
never dereferenced), and takes one beside them."""
import pytest

from moe_finalize_rmsnorm_gb300 import _abi
from moe_finalize_rmsnorm_gb300.build import build

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, CUDA, TIMEOUT, INVALID = range(9)
# buffers far apart
A, B, C, D, E, F, G, H = (0x100000000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def gemm():
    build()

    def call(x=A, xr=10, xs=32, sc=B, scs=16, ri=C, w=D, ws=32, we=32 * 32, wsc=E, wscs=16,
             wsce=16 * 32, fmt=0, f=F, off=G, out=H, odt=0, os=32, rows=10, E_=4, n=32, k=64):
        return _abi.lib().moe_grouped_gemm_fp4(x, xr, xs, sc, scs, ri, w, ws, we, wsc, wscs, wsce,
                                               fmt, f, off, out, odt, os, rows, E_, n, k, None)
    return call


OUT = 10 * 32 * 2   # bytes of the output


@pytest.mark.parametrize("at,size", [(A, 10 * 32), (B, 9 * 16 + 2), (C, 40), (D, 4 * 1024),
                                     (E, 3 * 512 + 31 * 16 + 2), (F, 16), (G, 20)])
def test_output_over_an_input(gemm, at, size):
    last = (size - 1) // 16 * 16   # the last 16 bytes that begin inside
    for out in (at, at + last, at - OUT + 16):
        assert gemm(out=out) == ALIGN, hex(out)
        assert gemm(out=out, odt=1) == ALIGN
    assert gemm(out=at - 2 * OUT + 16, odt=1) == ALIGN


def test_strided_experts(gemm):
    """Experts' matrices apart from each other, by whole rows or not."""
    for apart in (64 * 32, 64 * 32 + 16):
        assert gemm(we=apart, out=D + 3 * apart + 31 * 32) == ALIGN
        assert gemm(we=apart, out=D + apart) == ALIGN


def test_rows_far_apart(gemm):
    """Ends of rows that 64 bits do not hold."""
    assert gemm(xr=2 ** 31 - 1025, xs=2 ** 36 - 16, out=A + 32) == ALIGN


def test_without_index_factor_and_offsets(gemm):
    """What is not there has no place."""
    one = dict(E_=1, off=None, f=None, ri=None)
    assert gemm(**one, out=A) == ALIGN and gemm(**one, out=D + 31 * 32) == ALIGN


@pytest.mark.gpu
def test_side_by_side(cuda_lib):
    """Columns of one buffer's rows: the rows' bytes and the results lie between each other,
    and share none."""
    import torch
    import fp4_common as fp4
    rows, n, k = 40, 32, 64
    q, s = cuda_lib.moe_fp4_empty((rows,), k, fp4.MX)
    cuda_lib.moe_quantize_fp4(torch.randn((rows, k), device="cuda"), q, s)
    w, ws = cuda_lib.moe_fp4_empty((1, n), k, fp4.MX)
    w.random_(0, 256)
    ws.view(torch.uint8).fill_(127)
    want = cuda_lib.moe_grouped_gemm_fp4(q, s, w, ws, None, torch.empty((rows, n), device="cuda"))
    whole = torch.zeros((rows, 32 + 4 * n), dtype=torch.uint8, device="cuda")
    x, out = whole[:, :32], whole.view(torch.float32)[:, 8:]
    x.copy_(q)
    cuda_lib.moe_grouped_gemm_fp4(x, s, w, ws, None, out)
    assert torch.equal(out, want) and torch.equal(x, q)
