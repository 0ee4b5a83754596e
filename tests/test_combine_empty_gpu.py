"""Gradients of no rows or no tokens, with tensors that have no elements."""
import pytest
import torch

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.mark.parametrize("rows", [0, 3])
def test_no_tokens(cuda_lib, rows):
    none = torch.empty((0, 64), device="cuda")
    p = torch.ones((rows, 64), device="cuda")
    w = torch.empty((0, 2), device="cuda")
    idx = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    gp = torch.full((rows, 64), NAN, device="cuda")
    gw = torch.empty((0, 2), device="cuda")
    back = cuda_lib.moe_combine_backward
    assert back(none, p, None, idx, None, gw)[1] is gw      # as of a weighted way in
    assert back(none, None, w, idx, gp, None)[0] is gp
    back(none, p, w, idx, gp, gw)
    assert gp.isnan().all()                                 # rows that no entry names


def test_no_rows(cuda_lib):
    none = torch.empty((0, 64), device="cuda")
    dy = torch.ones((4, 64), device="cuda")
    w = torch.ones((4, 2), device="cuda")
    idx = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    gw = torch.full((4, 2), NAN, device="cuda")
    back = cuda_lib.moe_combine_backward
    assert back(dy, None, w, idx, none.clone(), None)[1] is None
    back(dy, none, None, idx, None, gw)
    assert (gw == 0).all()
    gw.fill_(NAN)
    back(dy, none, w, idx, none.clone(), gw)
    assert (gw == 0).all()
