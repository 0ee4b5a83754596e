"""Every product as the first work on the device of a thread, which has no context yet."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

MX = torch.float8_e8m0fnu


def operands(mf, rows, E=2, n=64, k=512):
    """name: (call, output's shape) of every operation, with nothing left to allocate."""
    off = torch.tensor([0, rows // 2, rows], device="cuda").int()
    x = torch.randn((rows, k), device="cuda").bfloat16()
    dy = torch.randn((rows, n), device="cuda").bfloat16()
    w = torch.randn((E, n, k), device="cuda").bfloat16()
    q, s = mf.moe_fp4_empty((rows,), k, MX)
    mf.moe_quantize_fp4(x, q, s)
    w4, w4s = mf.moe_fp4_empty((E, n), k, MX)
    w4.random_(0, 256)
    w4s.view(torch.uint8).fill_(125)
    w_int4 = torch.randint(0, 256, (E, n, k // 2), device="cuda").to(torch.uint8)
    int4_scales = torch.rand((E, n, k // 32), device="cuda").bfloat16()
    return {
        "gemm": (lambda o: mf.moe_grouped_gemm(x, w, off, o), (rows, n)),
        "dgrad": (lambda o: mf.moe_grouped_gemm_dgrad(dy, w, off, o), (rows, k)),
        "wgrad": (lambda o: mf.moe_grouped_gemm_wgrad(dy, x, off, o), (E, n, k)),
        "int4": (lambda o: mf.moe_grouped_gemv_int4(x, w_int4, int4_scales, off, o), (rows, n)),
        "fp4": (lambda o: mf.moe_grouped_gemm_fp4(q, s, w4, w4s, off, o), (rows, n)),
        "dequantize": (lambda o: mf.moe_dequantize_fp4(q, s, o), (rows, k)),
    }


@pytest.mark.parametrize("rows", [2, 300])
@pytest.mark.parametrize("name", ["gemm", "dgrad", "wgrad", "int4", "fp4", "dequantize"])
def test_a_threads_first_call(cuda_lib, name, rows):
    call, shape = operands(cuda_lib, rows)[name]
    here, there = (torch.full(shape, float("nan"), device="cuda") for _ in range(2))
    call(here)
    torch.cuda.synchronize()
    failed = []

    def run():
        try:
            call(there)
        except Exception as e:   # reported below: a thread's is only printed
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert torch.equal(here, there) and not here.isnan().any()
