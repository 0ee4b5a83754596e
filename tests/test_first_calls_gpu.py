"""First calls of several families of operations at once, from threads of a fresh process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
import moe_finalize_rmsnorm_gb300 as mf

E, rows, n, k = 4, 400, 264, 512
off = torch.arange(E + 1, device="cuda").int() * (rows // E)
x = torch.randn((rows, k), device="cuda").bfloat16()
w = torch.randn((E, n, k), device="cuda").bfloat16()
w4, w4s = mf.moe_fp4_empty((E, n), k, torch.float8_e4m3fn)
w4.random_(0, 256)
w4s.view(torch.uint8).fill_(0x38)
q, qs = mf.moe_fp4_empty((rows,), k, torch.float8_e4m3fn)
ids = torch.randint(0, E, (rows, 1), device="cuda", dtype=torch.int32)
torch.cuda.synchronize()


def bf16(out):
    return mf.moe_grouped_gemm(x, w, off, out)


def fp4(out):
    mf.moe_quantize_fp4(x, q, qs)
    return mf.moe_grouped_gemm_fp4(q, qs, w4, w4s, off, out)


def permutation(out):
    return mf.moe_expert_permutation(ids, E)[1]


calls = [bf16, fp4, permutation, bf16]
outs = [torch.empty((rows, n), device="cuda") for _ in calls]
streams = [torch.cuda.Stream() for _ in calls]
meet = threading.Barrier(len(calls), timeout=60)
got = [None] * len(calls)


def run(i):
    with torch.cuda.stream(streams[i]):
        meet.wait()
        got[i] = calls[i](outs[i]).clone()


threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
for i, call in enumerate(calls):
    assert torch.equal(call(torch.empty((rows, n), device="cuda")), got[i]), call.__name__
assert mf.device_status() == 0
print("same")
"""


def test_first_calls_at_once(cuda_lib):
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        assert r.stdout.strip() == "same"
