"""Expert offsets that do not fit their buffers: clamped to the rows, and without effect
where they do not ascend.  Every output lies between guard rows."""
import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf
from tests.test_experts_gpu import BF16, CANARY, FP32, int4_weights, randn

pytestmark = pytest.mark.gpu

GUARD = 8
N, K, EXPERTS = 40, 64, 4

DESCENDING = [[0, 50, 20, 70, 200], [-5, 10, 10, 2 ** 31 - 1, -2 ** 31], [90, 80, 70, 60, 50],
              [0, 30, 29, 29, 29], [1, 0, 0, 0, 0], [0, 0, 0, 5, 4]]
# as given, and what is left of them in `rows` rows
CLAMPED = [([3, 7, 7, 20, 30], lambda rows: [3, 7, 7, 20, min(30, rows)]),
           ([-7, -1, 9, 2 ** 31 - 1, 2 ** 31 - 1], lambda rows: [0, 0, 9, rows, rows]),
           ([2 ** 30] * 5, lambda rows: [rows] * 5),
           ([-2 ** 31] * 5, lambda rows: [0] * 5)]


def guarded(rows, width, dtype):
    buf = torch.full((rows + 2 * GUARD, width), CANARY, dtype=dtype, device="cuda")
    return buf, buf[GUARD:GUARD + rows]


def calls(rows):
    """(name, output width, call(offsets, output), weights [E, out, in], rows' values)"""
    w = randn((EXPERTS, N, K), 1)
    x, dy = randn((rows, K), 2), randn((rows, N), 3)
    index = torch.arange(rows, dtype=torch.int32, device="cuda")
    q, s, z, w4 = int4_weights(EXPERTS, N, K, 32, BF16, True, 4)
    return [
        ("forward", N, lambda o, y: mf.moe_grouped_gemm(x, w, o, y), w, x),
        ("gathered", N, lambda o, y: mf.moe_grouped_gemm(x, w, o, y, row_index=index), w, x),
        ("dgrad", K, lambda o, y: mf.moe_grouped_gemm_dgrad(dy, w, o, y), w.transpose(1, 2), dy),
        ("int4", N, lambda o, y: mf.moe_grouped_gemv_int4(x, q, s, o, y, zeros=z), w4, x),
        ("int4 gathered", N,
         lambda o, y: mf.moe_grouped_gemv_int4(x, q, s, o, y, zeros=z, row_index=index), w4, x),
    ]


# passes of 8, 16 and 32 rows in the 4-bit product; few rows and many in the others
@pytest.mark.parametrize("rows", [20, 64, 90, 300])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_offsets_that_do_not_ascend(cuda_lib, rows, dtype):
    """No row is written (lists that ascend once they are clamped are not meant)."""
    for name, width, call, _, _ in calls(rows):
        for bad in DESCENDING:
            clamped = [min(max(v, 0), rows) for v in bad]
            if clamped == sorted(clamped):
                continue
            buf, out = guarded(rows, width, dtype)
            call(torch.tensor(bad, dtype=torch.int32, device="cuda"), out)
            assert (buf == CANARY).all(), (name, bad)


@pytest.mark.parametrize("rows", [20, 64, 90, 300])
def test_offsets_beyond_the_rows(cuda_lib, rows):
    """The rows inside are right (to FP32 sums of at most 64 values), the others kept."""
    for name, width, call, w, x in calls(rows):
        for given, want in CLAMPED:
            buf, out = guarded(rows, width, FP32)
            call(torch.tensor(given, dtype=torch.int32, device="cuda"), out)
            ref = torch.full((rows, width), CANARY, dtype=torch.float64, device="cuda")
            mag = torch.zeros_like(ref)
            lo_hi = want(rows)
            for e, (lo, hi) in enumerate(zip(lo_hi[:-1], lo_hi[1:])):
                lo, hi = min(lo, rows), min(hi, rows)
                ref[lo:hi] = x[lo:hi].double() @ w[e].double().t()
                mag[lo:hi] = x[lo:hi].double().abs() @ w[e].double().abs().t()
            assert ((out.double() - ref).abs() <= 70 * 2.0 ** -23 * mag).all(), (name, given)
            assert (buf[:GUARD] == CANARY).all() and (buf[GUARD + rows:] == CANARY).all(), name


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_weight_gradients_stay_in_their_buffer(cuda_lib, gather, dtype):
    rows = 200
    x, dy = randn((rows, K), 2), randn((rows, N), 3)
    index = torch.arange(rows, dtype=torch.int32, device="cuda") if gather else None
    for given in DESCENDING + [g for g, _ in CLAMPED]:
        buf = torch.full((EXPERTS + 2, N, K), CANARY, dtype=dtype, device="cuda")
        mf.moe_grouped_gemm_wgrad(dy, x, torch.tensor(given, dtype=torch.int32, device="cuda"),
                                  buf[1:-1], row_index=index)
        assert (buf[0] == CANARY).all() and (buf[-1] == CANARY).all(), given


def test_many_experts_that_overlap(cuda_lib):
    """Every second expert claims all rows: half a million passes if they counted."""
    E, rows = 1024, 8192
    w = randn((E, 8, 32), 1)
    x = randn((rows, 32), 2)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    q, s, z, _ = int4_weights(E, 8, 32, 32, BF16, True, 4)
    for call in (lambda y: mf.moe_grouped_gemm(x, w, off, y),
                 lambda y: mf.moe_grouped_gemv_int4(x, q, s, off, y, zeros=z)):
        buf, out = guarded(rows, 8, BF16)
        call(out)
        assert (buf == CANARY).all()
