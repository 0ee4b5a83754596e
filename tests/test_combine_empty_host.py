"""Gradients of no rows or no tokens (CPU only).  A tensor without elements has a null
pointer, so it must not be taken for a gradient that is not wanted."""
import pytest

from moe_finalize_rmsnorm_gb300 import _abi
from moe_finalize_rmsnorm_gb300.build import build

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, CUDA, TIMEOUT, INVALID = range(9)
A, B, C, D, E, F = (0x100000000 * i for i in range(1, 7))


@pytest.fixture(scope="module")
def backward():
    build()

    def call(go=A, gs=64, p=B, rows=10, ps=64, w=C, wdt=1, idx=D, gp=E, gps=64, gw=F, gwdt=1, T=4,
             H=64, K=2):
        return _abi.lib().moe_combine_backward(go, 0, gs, p, 0, rows, ps, w, wdt, idx, gp, gps, gw,
                                               gwdt, T, H, K, None)
    return call


def test_no_tokens(backward):
    """Every operand with a token's dimension is empty; the rows may be there or not."""
    none = dict(T=0, go=None, w=None, idx=None)
    for rows, p in ((10, B), (0, None)):
        assert backward(**none, rows=rows, p=p, gp=None, gw=None) == OK   # grad_weights [0, K]
        assert backward(**none, rows=rows, p=p, gp=E if rows else None, gw=None) == OK
    assert backward(**none, p=None, gw=None) == OK


def test_no_rows(backward):
    """The rows' gradient alone has nothing to hold, with permuted or without it."""
    assert backward(rows=0, p=None, gp=None, gw=None) == OK
    assert backward(rows=0, p=B, gp=None, gw=None) == OK


def test_what_is_refused_stays_refused(backward):
    assert backward(gp=None, gw=None) == INVALID
    assert backward(rows=0, T=-1, gp=None, gw=None) == SHAPE
    assert backward(T=0, H=4, gp=None, gw=None) == UNSUP
    assert backward(T=0, gs=56, gp=None, gw=None) == SHAPE
    assert backward(rows=0, go=None, p=None, gp=None, gw=None) == NULL
    assert backward(rows=0, idx=None, p=None, gp=None, gw=None) == NULL
