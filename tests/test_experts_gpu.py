"""Parity of the expert-layer operations with their definitions in float64.

Tolerances.  A product of two BF16 values is exact in FP32.  Adding C of them in
FP32, in any order, with each addition rounded or truncated to 24 bits, is off by
at most C * 2^-23 * S, S the sum of the terms' magnitudes; the final rounding is
off by at most half a step of the output's type, 2^-8 (BF16) or 2^-24 (FP32) of
the value.  Where the result must be exactly zero S is zero, so is the bound.
"""
import itertools
import os
import random

import pytest
import torch

import moe_finalize_rmsnorm_gb300 as mf

pytestmark = pytest.mark.gpu

BF16, FP32, F64 = torch.bfloat16, torch.float32, torch.float64
ROUND = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
CANARY = 7.25  # exact in BF16; what untouched rows hold


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(shape, seed, dtype=BF16):
    return torch.randn(shape, generator=gen(seed)).to(dtype).cuda()


def within(got, ref, mag, terms, dtype):
    """|got - ref| <= rounding + accumulation; NaN and infinity must agree."""
    got, ref, mag = got.double(), ref.double(), mag.double()
    bad = torch.isnan(got) != torch.isnan(ref)
    assert not bad.any(), f"NaN disagrees at {bad.nonzero()[:4].tolist()}"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf])
    ok = torch.isfinite(ref)
    acc = terms * 2.0 ** -23 * mag
    tol = acc + ROUND[dtype] * (ref.abs() + acc)
    off = ((got - ref).abs() > tol) & ok
    assert not off.any(), (
        f"{int(off.sum())} of {off.numel()} outside, first at {off.nonzero()[:4].tolist()}: "
        f"{got[off][:4].tolist()} against {ref[off][:4].tolist()}, bound {tol[off][:4].tolist()}")


def offsets_of(sizes):
    return torch.tensor([0, *itertools.accumulate(sizes)], dtype=torch.int32).cuda()


def gathered(x, index, rows):
    """float64 rows that the product reads: zeros where the index is outside."""
    if index is None:
        return x[:rows].double()
    i = index.long()
    ok = (i >= 0) & (i < x.shape[0])
    r = x[i.clamp(0, x.shape[0] - 1)].double()
    r[~ok] = 0
    return r


# ---------------------------------------------------------------------------
# permutation by expert

def permutation_ref(ids, experts):
    """Offsets, slot -> row and row -> token by a walk over the slots."""
    T, K = ids.shape
    flat = ids.flatten().tolist()
    of = [[s for s, e in enumerate(flat) if e == x] for x in range(experts)]
    offsets = [0, *itertools.accumulate(len(o) for o in of)]
    rows = [s for o in of for s in o]
    pos = [-1] * (T * K)
    for r, s in enumerate(rows):
        pos[s] = r
    tok = [s // K for s in rows] + [-1] * (T * K - len(rows))
    as_i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return as_i32(offsets), as_i32(pos).view(T, K), as_i32(tok)


def check_permutation(ids, experts, packed=False, words=None):
    off, idx, tok = mf.moe_expert_permutation((ids if words is None else words).cuda(), experts,
                                              packed=packed)
    ref = permutation_ref(ids, experts)
    for got, want, name in zip((off, idx, tok), ref, ("offsets", "idx", "row_to_token")):
        assert torch.equal(got.cpu(), want), name


@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 8), (3, 5, 7), (32, 8, 128), (33, 8, 1024),
                                   (257, 3, 1000), (1000, 6, 64), (4096, 8, 60), (5003, 7, 33)])
def test_permutation(cuda_lib, T, K, E):
    ids = torch.randint(0, E, (T, K), generator=gen(T + E), dtype=torch.int32)
    check_permutation(ids, E)
    # a fifth of the slots without an expert, on both sides of the range
    drop = torch.rand((T, K), generator=gen(1)) < 0.2
    ids[drop] = torch.where(torch.rand((T, K), generator=gen(2)) < 0.5, -1, E)[drop].int()
    check_permutation(ids, E)


@pytest.mark.parametrize("T,K,E", [(300, 8, 16), (40000, 8, 256)])
def test_permutation_extremes(cuda_lib, T, K, E):
    one = torch.full((T, K), E - 1, dtype=torch.int32)
    none = torch.full((T, K), -1, dtype=torch.int32)
    far = torch.full((T, K), 2 ** 31 - 1, dtype=torch.int32)
    turns = (torch.arange(T * K, dtype=torch.int32) % E).view(T, K)
    for ids in (one, none, far, turns, turns.flip(0).contiguous()):
        off, idx, tok = mf.moe_expert_permutation(ids.cuda(), E)
        live = (ids >= 0) & (ids < E)
        key = torch.where(live, ids, E).flatten()
        order = key.argsort(stable=True)
        n = int(live.sum())
        assert torch.equal(off.cpu(), torch.searchsorted(
            key[order], torch.arange(E + 1, dtype=torch.int32)).int())
        want = torch.full((T * K,), -1, dtype=torch.int32)
        want[order[:n]] = torch.arange(n, dtype=torch.int32)
        assert torch.equal(idx.cpu().flatten(), want)
        tokens = torch.full((T * K,), -1, dtype=torch.int32)
        tokens[:n] = (order[:n] // K).int()
        assert torch.equal(tok.cpu(), tokens)


@pytest.mark.parametrize("slots", [4095, 4096, 4097, 5120, 8191, 8192, 8193, 10239, 10240, 131071, 131072, 131073, 311296,
                                   400001])
@pytest.mark.parametrize("E", [1, 7, 1024])
def test_permutation_at_the_edges_of_its_launches(cuda_lib, slots, E):
    """Where one CTA hands over to several, and the chunks' and the cluster's sizes change."""
    ids = torch.randint(-1, E + 1, (slots, 1), generator=gen(slots), dtype=torch.int32)
    off, idx, tok = mf.moe_expert_permutation(ids.cuda(), E)
    live = (ids >= 0) & (ids < E)
    key = torch.where(live, ids, E).flatten()
    order = key.argsort(stable=True).int()
    n = int(live.sum())
    counts = torch.bincount(key, minlength=E + 1)[:E]
    assert torch.equal(off.cpu()[1:], counts.cumsum(0).int()) and off[0] == 0
    assert torch.equal(tok.cpu()[:n], order[:n]) and (tok.cpu()[n:] == -1).all()
    want = torch.full((slots,), -1, dtype=torch.int32)
    want[order[:n].long()] = torch.arange(n, dtype=torch.int32)
    assert torch.equal(idx.cpu().flatten(), want)


def test_permutation_of_packed_words(cuda_lib):
    # ids above 32767 make negative words; 65535 is outside any range
    ids = torch.randint(0, 1000, (400, 8), generator=gen(3), dtype=torch.int32)
    ids[5, 3], ids[6, 0], ids[7, 7] = 65535, 40000, 1000
    words = ((ids.long() << 16) | 0xBF80).to(torch.int64)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    check_permutation(ids, 1000, packed=True, words=words)


def test_permutation_of_no_tokens(cuda_lib):
    off, idx, tok = mf.moe_expert_permutation(
        torch.empty((0, 8), dtype=torch.int32, device="cuda"), 16)
    assert off.tolist() == [0] * 17 and idx.shape == (0, 8) and tok.numel() == 0


def test_permutation_writes_the_given_tensors(cuda_lib):
    ids = torch.randint(0, 9, (50, 4), generator=gen(4), dtype=torch.int32).cuda()
    mine = (torch.empty(10, dtype=torch.int32, device="cuda"),
            torch.empty((50, 4), dtype=torch.int32, device="cuda"),
            torch.empty(200, dtype=torch.int32, device="cuda"))
    got = mf.moe_expert_permutation(ids, 9, expert_offsets=mine[0], expanded_idx=mine[1],
                                    row_tokens=mine[2])
    assert all(a is b for a, b in zip(got, mine))
    for a, b in zip(mine, mf.moe_expert_permutation(ids, 9)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# the gradient of the gather

@pytest.mark.parametrize("in_dtype,out_dtype", list(itertools.product((BF16, FP32), repeat=2)))
@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (1, 8, 4096), (77, 6, 264), (500, 8, 1000),
                                   (19, 32, 72), (3, 2, 16384)])
def test_row_sum(cuda_lib, T, K, H, in_dtype, out_dtype):
    rows = T * K + 5
    buf = randn((rows, H + 8), T + H, in_dtype)
    buf[:, H:] = float("nan")            # columns behind the row
    p = buf[:, :H]
    idx = torch.randint(-2, rows - 3, (T, K), generator=gen(T), dtype=torch.int32)
    idx[0, 0] = rows + 10                # outside on either side: contributes nothing
    p[rows - 3:] = float("nan")          # rows that no slot selects
    out = torch.full((T, H), CANARY, dtype=out_dtype, device="cuda")
    assert mf.moe_permuted_row_sum(p, idx.cuda(), out) is out
    ref = gathered(p, idx.flatten().cuda(), 0).view(T, K, H)
    within(out, ref.sum(1), ref.abs().sum(1), K, out_dtype)


def test_row_sum_same_row_twice_and_non_finite(cuda_lib):
    p = randn((4, 64), 1)
    p[2, 5], p[3, 7] = float("inf"), float("nan")
    idx = torch.tensor([[0, 0, 0], [2, 1, -1], [3, -1, 9], [-1, -1, -1]], dtype=torch.int32).cuda()
    out = torch.empty((4, 64), dtype=FP32, device="cuda")
    mf.moe_permuted_row_sum(p, idx, out)
    ref = gathered(p, idx.flatten(), 0).view(4, 3, 64)
    within(out, ref.sum(1), ref.abs().sum(1), 3, FP32)
    assert (out[3] == 0).all()


def test_row_sum_of_no_rows(cuda_lib):
    out = torch.full((3, 64), CANARY, dtype=BF16, device="cuda")
    mf.moe_permuted_row_sum(torch.empty((0, 64), dtype=BF16, device="cuda"),
                            torch.zeros((3, 2), dtype=torch.int32, device="cuda"), out)
    assert (out == 0).all()


# ---------------------------------------------------------------------------
# grouped products

SIZES = {
    "one_row": [1],
    "one_token": [1, 0, 1, 1, 0, 0, 1, 1],
    "few": [3, 0, 8, 1, 17, 2],
    "tile_edges": [127, 128, 0, 129, 1, 255, 256, 257],
    "skewed": [700, 0, 0, 5, 61, 1, 33, 0],
    "none": [0, 0, 0],
}
WIDTHS = [(8, 8), (24, 72), (136, 200), (264, 1000), (512, 256), (1000, 520)]


def weights(E, n, k, seed, pad_k=0, pad_n=0):
    """A [E, n, k] view with padded rows and experts; the padding is NaN."""
    buf = torch.full((E, n + pad_n, k + pad_k), float("nan"), dtype=BF16, device="cuda")
    w = buf[:, :n, :k]
    w.copy_(randn((E, n, k), seed) * k ** -0.5)
    return w


def padded(rows, width, seed, pad):
    buf = torch.full((rows, width + pad), float("nan"), dtype=BF16, device="cuda")
    v = buf[:, :width]
    v.copy_(randn((rows, width), seed))
    return v


def check_rows(out, sizes, groups, terms, dtype):
    """out's rows against (result, magnitudes) per expert; rows behind the last
    one keep the canary."""
    lo = 0
    for m, (ref, mag) in zip(sizes, groups):
        within(out[lo:lo + m], ref, mag, terms, dtype)
        lo += m
    assert (out[lo:] == CANARY).all(), "rows behind the last were written"


def check_forward(sizes, n, k, dtype, *, gather=False, pad=0, extra=3, seed=0):
    E, rows = len(sizes), sum(sizes) + extra
    w = weights(E, n, k, seed + 1, pad, 1 if pad else 0)
    x = padded(max(rows, 1), k, seed + 2, pad)
    index = None
    if gather:
        x = padded(37, k, seed + 2, pad)
        index = torch.randint(0, 37, (rows,), generator=gen(seed), dtype=torch.int32)
        index[::11] = torch.tensor([-1, 37, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(
            rows)[:index[::11].numel()]
        index = index.cuda()
    else:
        x[sum(sizes):] = float("nan")    # rows of no expert
    buf = torch.full((rows, n + pad), CANARY, dtype=dtype, device="cuda")
    out = buf[:, :n]
    assert mf.moe_grouped_gemm(x, w, offsets_of(sizes), out, row_index=index) is out
    a = gathered(x, index, rows)
    groups, lo = [], 0
    for e, m in enumerate(sizes):
        r, we = a[lo:lo + m], w[e].double()
        groups.append((r @ we.t(), r.abs() @ we.abs().t()))
        lo += m
    check_rows(out, sizes, groups, k, dtype)
    assert (buf[:, n:] == CANARY).all(), "columns behind the row were written"


@pytest.mark.parametrize("n,k", WIDTHS)
@pytest.mark.parametrize("which", list(SIZES))
def test_forward(cuda_lib, which, n, k):
    check_forward(SIZES[which], n, k, BF16)
    check_forward(SIZES[which], n, k, FP32, pad=8, seed=10)
    check_forward(SIZES[which], n, k, BF16, gather=True, pad=16, seed=20)


@pytest.mark.parametrize("sizes,n,k", [([4], 2048, 4096), ([1, 2, 0, 1], 4096, 7168),
                                       ([300, 0, 211], 1416, 2200), ([2000], 256, 2048),
                                       ([40] * 40, 128, 192)])
def test_forward_wide(cuda_lib, sizes, n, k):
    check_forward(sizes, n, k, BF16)
    check_forward(sizes, n, k, FP32, gather=True, seed=5)


@pytest.mark.parametrize("sizes", [[64], [65], [60, 1, 2, 1], [16, 17, 0, 31], [0, 0, 64, 0],
                                   [2] * 128, [256] + [0] * 127, [253] + [0] * 128, [1] * 64])
@pytest.mark.parametrize("n,k", [(136, 200), (1000, 1416)])
def test_forward_where_the_few_rows_kernel_ends(cuda_lib, sizes, n, k):
    for extra in (0, 1):
        check_forward(sizes, n, k, FP32, extra=extra)
        check_forward(sizes, n, k, BF16, gather=True, pad=8, extra=extra, seed=3)


def test_few_rows_with_long_sums(cuda_lib):
    """As test_fp32_sums_over_long_dimensions, at the sizes of the other kernel."""
    n, k = 264, 16384
    w, x = weights(2, n, k, 1), padded(20, k, 2, 0)
    out = torch.empty((20, n), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm(x, w, offsets_of([13, 7]), out)
    for e, sl in ((0, slice(0, 13)), (1, slice(13, 20))):
        within(out[sl], x[sl].double() @ w[e].double().t(),
               x[sl].double().abs() @ w[e].double().abs().t(), 2 * (40 + k // 640 + 13), FP32)


def test_forward_many_experts(cuda_lib):
    sizes = [(7 * e) % 5 if e % 3 else 0 for e in range(1024)]
    check_forward(sizes, 64, 64, BF16)
    sizes[500] = 600
    check_forward(sizes, 64, 64, FP32)


def check_dgrad(sizes, n, k, dtype, *, pad=0, extra=3, seed=0):
    E, rows = len(sizes), sum(sizes) + extra
    w = weights(E, n, k, seed + 1, pad, 1 if pad else 0)
    dy = padded(rows, n, seed + 2, pad)
    dy[sum(sizes):] = float("nan")
    buf = torch.full((rows, k + pad), CANARY, dtype=dtype, device="cuda")
    out = buf[:, :k]
    assert mf.moe_grouped_gemm_dgrad(dy, w, offsets_of(sizes), out) is out
    groups, lo = [], 0
    for e, m in enumerate(sizes):
        r, we = dy[lo:lo + m].double(), w[e].double()
        groups.append((r @ we, r.abs() @ we.abs()))
        lo += m
    check_rows(out, sizes, groups, n, dtype)
    assert (buf[:, k:] == CANARY).all()


@pytest.mark.parametrize("n,k", WIDTHS)
@pytest.mark.parametrize("which", list(SIZES))
def test_dgrad(cuda_lib, which, n, k):
    check_dgrad(SIZES[which], n, k, BF16)
    check_dgrad(SIZES[which], n, k, FP32, pad=8, seed=10)


def check_wgrad(sizes, n, k, dtype, *, gather=False, accumulate=False, pad=0, extra=3, seed=0):
    E, rows = len(sizes), sum(sizes) + extra
    dy = padded(rows, n, seed + 1, pad)
    x = padded(rows, k, seed + 2, pad)
    dy[sum(sizes):] = float("nan")       # rows of no expert, right behind the last expert's
    index = None
    if gather:
        x = padded(37, k, seed + 2, pad)
        index = torch.randint(0, 37, (rows,), generator=gen(seed), dtype=torch.int32)
        index[::11] = -1
        index[5::13] = 37
        index = index.cuda()
    else:
        x[sum(sizes):] = float("nan")
    base = randn((E, n, k), seed + 3, dtype)
    out = base.clone()
    assert mf.moe_grouped_gemm_wgrad(dy, x, offsets_of(sizes), out, row_index=index,
                                     accumulate=accumulate) is out
    a = gathered(x, index, rows)
    lo = 0
    for e, m in enumerate(sizes):
        g, r = dy[lo:lo + m].double(), a[lo:lo + m]
        ref, mag = g.t() @ r, g.abs().t() @ r.abs()
        if accumulate:
            ref, mag = ref + base[e].double(), mag + base[e].double().abs()
        within(out[e], ref, mag, m + 1, dtype)
        lo += m


@pytest.mark.parametrize("n,k", WIDTHS)
@pytest.mark.parametrize("which", list(SIZES))
def test_wgrad(cuda_lib, which, n, k):
    check_wgrad(SIZES[which], n, k, BF16, pad=8)
    check_wgrad(SIZES[which], n, k, FP32, gather=True, seed=10)
    check_wgrad(SIZES[which], n, k, FP32, accumulate=True, seed=20)
    check_wgrad(SIZES[which], n, k, BF16, gather=True, accumulate=True, pad=16, seed=30)


def test_weights_gradient_of_no_rows(cuda_lib):
    dy = torch.empty((0, 24), dtype=BF16, device="cuda")
    x = torch.empty((0, 40), dtype=BF16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    for dtype in (BF16, FP32):
        dw = torch.full((3, 24, 40), CANARY, dtype=dtype, device="cuda")
        mf.moe_grouped_gemm_wgrad(dy, x, off, dw, accumulate=True)
        assert (dw == CANARY).all()
        mf.moe_grouped_gemm_wgrad(dy, x, off, dw)
        assert (dw == 0).all()


def test_every_other_expert(cuda_lib):
    """A weight view that skips experts and starts inside its buffer."""
    sizes, n, k = [5, 0, 130, 9], 136, 264
    w = weights(9, n, k, 1, 8, 1)[1::2]
    x = padded(144, k, 2, 8)
    out = torch.empty((144, n), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm(x, w, offsets_of(sizes), out)
    lo = 0
    for e, m in enumerate(sizes):
        r, we = x[lo:lo + m].double(), w[e].double()
        within(out[lo:lo + m], r @ we.t(), r.abs() @ we.abs().t(), k, FP32)
        lo += m


@pytest.mark.parametrize("n,k", [(65536, 8), (8, 65536), (40000, 72)])
def test_wide_and_flat_matrices(cuda_lib, n, k):
    check_forward([3, 0, 20], n, k, FP32)
    check_dgrad([3, 0, 20], n, k, BF16)
    check_wgrad([3, 0, 20], n, k, BF16)


def test_fp32_sums_over_long_dimensions(cuda_lib):
    """FP32 results are summed outside the tensor cores every 640 values.  Inside, each
    of the 40 products of 16 values that are added to one sum loses at most 2^-22 of
    the running magnitude (two truncated bits), outside each addition 2^-24: C values
    lose (40 + C / 640) * 2^-22 of S, not C * 2^-23."""
    n, k, rows = 264, 16384, 300
    w, x = weights(1, n, k, 1), padded(rows, k, 2, 0)
    off = offsets_of([rows])
    out = torch.empty((rows, n), dtype=FP32, device="cuda")
    dw = torch.empty((1, n, 264), dtype=FP32, device="cuda")
    index = torch.arange(rows, dtype=torch.int32, device="cuda")
    terms = 2 * (40 + k // 640 + 1)
    for ix in (None, index):
        mf.moe_grouped_gemm(x, w, off, out, row_index=ix)
        within(out, x.double() @ w[0].double().t(), x.double().abs() @ w[0].double().abs().t(),
               terms, FP32)
        rel = (out.double() - x.double() @ w[0].double().t()).norm() / out.double().norm()
        assert rel < 1e-6, rel
    many = 9000
    dy, xx = padded(many, n, 3, 0), padded(many, 264, 4, 0)
    off = offsets_of([many])
    index = torch.arange(many, dtype=torch.int32, device="cuda")
    terms = 2 * (40 + many // 640 + 1)
    for ix in (None, index):
        mf.moe_grouped_gemm_wgrad(dy, xx, off, dw, row_index=ix)
        within(dw[0], dy.double().t() @ xx.double(), dy.double().abs().t() @ xx.double().abs(),
               terms, FP32)


def test_non_finite_rows_stay_in_their_expert(cuda_lib):
    """A NaN row touches its own output row, and its own expert's gradient only."""
    sizes, n, k = [70, 3, 90], 136, 200
    x, dy = padded(163, k, 1, 0), padded(163, n, 2, 0)
    x[71], dy[71] = float("nan"), float("inf")
    off = offsets_of(sizes)
    w = weights(3, n, k, 3)
    out = torch.empty((163, n), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm(x, w, off, out)
    dx = torch.empty((163, k), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm_dgrad(dy, w, off, dx)
    dw = torch.empty((3, n, k), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm_wgrad(dy, x, off, dw)
    clean = torch.arange(163, device="cuda") != 71
    assert torch.isnan(out[71]).all() and torch.isfinite(out[clean]).all()
    assert not torch.isfinite(dx[71]).any() and torch.isfinite(dx[clean]).all()
    assert torch.isnan(dw[1]).all() and torch.isfinite(dw[0]).all() and torch.isfinite(dw[2]).all()


def test_offsets_that_do_not_ascend_stay_in_bounds(cuda_lib):
    """The values are unspecified; nothing outside the rows is written."""
    n, k = 64, 128
    x, w = padded(100, k, 1, 0), weights(4, n, k, 2)
    for bad in ([0, 50, 20, 70, 200], [-5, 10, 10, 2 ** 31 - 1, -2 ** 31], [90, 80, 70, 60, 50],
                [2 ** 30] * 5):
        buf = torch.full((104, n), CANARY, dtype=BF16, device="cuda")
        dw = torch.full((5, n, k), CANARY, dtype=BF16, device="cuda")
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        mf.moe_grouped_gemm(x, w, off, buf[:100])
        mf.moe_grouped_gemm_wgrad(buf[:100], x, off, dw[:4])
        torch.cuda.synchronize()
        assert (buf[100:] == CANARY).all() and (dw[4] == CANARY).all()


# ---------------------------------------------------------------------------
# 4-bit weights

def int4_weights(E, n, k, group, scale_dtype, zeros, seed):
    g = gen(seed)
    q = torch.randint(0, 256, (E, n, k // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand((E, n, k // group), generator=g) * 0.02 + 0.001).to(scale_dtype)
    z = torch.randint(0, 16, (E, n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    nib = torch.stack((q & 15, q >> 4), dim=-1).flatten(2).double()
    zz = 8.0 if z is None else z.double().repeat_interleave(group, 2)
    w = (nib - zz) * s.double().repeat_interleave(group, 2)
    return q.cuda(), s.cuda(), None if z is None else z.cuda(), w.cuda()


def check_int4(sizes, n, k, group, dtype, *, scale_dtype=BF16, zeros=False, gather=False, pad=0,
               dense=False, seed=0):
    E, extra = len(sizes), 0 if dense else 3
    rows = sum(sizes) + extra
    q, s, z, w = int4_weights(E, n, k, group, scale_dtype, zeros, seed)
    x = padded(rows, k, seed + 2, pad)
    index = None
    if gather:
        x = padded(9, k, seed + 2, pad)
        index = torch.randint(0, 9, (rows,), generator=gen(seed), dtype=torch.int32)
        index[2::7] = -1
        index[3::11] = 9
        index = index.cuda()
    elif not dense:
        x[sum(sizes):] = float("nan")
    buf = torch.full((rows, n + pad), CANARY, dtype=dtype, device="cuda")
    out = buf[:, :n]
    off = None if dense else offsets_of(sizes)
    assert mf.moe_grouped_gemv_int4(x, q, s, off, out, zeros=z, row_index=index) is out
    a = gathered(x, index, rows)
    groups, lo = [], 0
    for e, m in enumerate(sizes):
        r = a[lo:lo + m]
        groups.append((r @ w[e].t(), r.abs() @ w[e].abs().t()))
        lo += m
    check_rows(out, sizes, groups, k + 2 * k // group, dtype)
    assert (buf[:, n:] == CANARY).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("sizes", [[1], [2, 0, 1, 1], [8, 7, 9, 0, 16, 17], [33, 1, 64, 65],
                                   [5, 5], [6, 5], [100, 0, 0, 0, 1]])
def test_int4(cuda_lib, sizes, group):
    for i, (n, k) in enumerate(((1, group), (7, 3 * group), (33, 8 * group), (100, 640),
                                (256, 1152))):
        check_int4(sizes, n, k, group, BF16, seed=i)
        check_int4(sizes, n, k, group, FP32, scale_dtype=FP32, zeros=True, seed=i + 10)
        check_int4(sizes, n, k, group, BF16, zeros=True, gather=True, pad=8, seed=i + 20)


@pytest.mark.parametrize("rows", [1, 3, 8, 9, 24, 25, 40, 64, 65])
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (1001, 4096, 128), (515, 7168, 64),
                                       (64, 16384, 32)])
def test_int4_dense(cuda_lib, rows, n, k, group):
    check_int4([rows], n, k, group, BF16, dense=True, zeros=True)
    check_int4([rows], n, k, group, FP32, dense=True, scale_dtype=FP32, seed=3)


@pytest.mark.parametrize("group,k", [(32, 512), (64, 512), (128, 512), (32, 96), (128, 384)])
def test_int4_scales_at_any_word(cuda_lib, group, k):
    """Scales and zeros that start at any 4-byte boundary."""
    sizes, n = [3, 20, 1], 45
    for scale_dtype, skip in ((BF16, 2), (BF16, 6), (FP32, 1), (FP32, 3)):
        q, s, z, w = int4_weights(3, n, k, group, scale_dtype, True, 1)
        sbuf = torch.empty(s.numel() + skip, dtype=scale_dtype, device="cuda")
        sv = sbuf[skip:].view(s.shape).copy_(s)
        zbuf = torch.empty(z.numel() + 4, dtype=torch.uint8, device="cuda")
        zv = zbuf[4:].view(z.shape).copy_(z)
        x = padded(24, k, 2, 0)
        out = torch.empty((24, n), dtype=FP32, device="cuda")
        mf.moe_grouped_gemv_int4(x, q, sv, offsets_of(sizes), out, zeros=zv)
        lo = 0
        for e, m in enumerate(sizes):
            r = x[lo:lo + m].double()
            within(out[lo:lo + m], r @ w[e].t(), r.abs() @ w[e].abs().t(), k + 2 * k // group, FP32)
            lo += m


def test_int4_every_nibble_and_zero(cuda_lib):
    """All 256 pairs of nibble and zero point, exactly (one value a row of x)."""
    k, n = 256, 512
    q = torch.arange(256, dtype=torch.int32)
    nib = (q % 16).repeat(n, 1)                         # column c holds c % 16
    packed = (nib[:, 0::2] | nib[:, 1::2] << 4).to(torch.uint8).view(1, n, k // 2).cuda()
    zeros = (torch.arange(n * 8) // 8 % 16).to(torch.uint8).view(1, n, 8).cuda()
    scales = torch.ones((1, n, 8), dtype=FP32, device="cuda")
    x = torch.zeros((16, k), dtype=BF16, device="cuda")
    x[torch.arange(16), torch.arange(16) + 48] = 1.0    # row r picks column 48 + r
    out = torch.empty((16, n), dtype=FP32, device="cuda")
    mf.moe_grouped_gemv_int4(x, packed, scales, None, out, zeros=zeros)
    want = torch.arange(16).view(16, 1) - (torch.arange(n) % 16).view(1, n)
    assert torch.equal(out.cpu(), want.float())


def test_int4_many_experts(cuda_lib):
    sizes = [(5 * e) % 4 if e % 2 else 0 for e in range(1024)]
    check_int4(sizes, 24, 128, 64, FP32, zeros=True)


def test_int4_non_finite_rows(cuda_lib):
    """A NaN row, and an infinite scale, stay where they belong."""
    q, s, z, _ = int4_weights(2, 40, 256, 64, BF16, True, 1)
    x = padded(6, 256, 2, 0)
    x[1] = float("nan")
    s[1, 3, 2] = float("inf")
    out = torch.empty((6, 40), dtype=FP32, device="cuda")
    mf.moe_grouped_gemv_int4(x, q, s, offsets_of([3, 3]), out, zeros=z)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[1] = True
    want[3:, 3] = True
    assert torch.equal(bad, want)


# ---------------------------------------------------------------------------
# seeded random configurations

def draw_sizes(rng):
    E = rng.choice([1, 2, 3, 7, 16, 40, 130, 600])
    kind = rng.choice(["even", "skewed", "sparse", "one"])
    total = rng.choice([0, 1, 5, 64, 65, 200, 1000, 3000])
    if kind == "one":
        sizes = [0] * E
        sizes[rng.randrange(E)] = total
        return sizes
    w = {"even": [1.0] * E, "skewed": [(1 + e) ** -1.5 for e in range(E)],
         "sparse": [rng.random() < 0.2 for _ in range(E)]}[kind]
    w = w if sum(w) else [1.0] * E
    sizes = [0] * E
    for _ in range(total):
        sizes[rng.choices(range(E), w)[0]] += 1
    return sizes


@pytest.mark.parametrize("seed", range(int(os.environ.get("MF_FUZZ_SEEDS", "24"))))
def test_random_grouped_products(cuda_lib, seed):
    rng = random.Random(seed)
    sizes = draw_sizes(rng)
    widest = 2000 if len(sizes) < 100 else 300
    n, k = (8 * rng.randint(1, widest // 8) for _ in range(2))
    dtype = rng.choice([BF16, FP32])
    pad, extra = rng.choice([0, 8, 40]), rng.choice([0, 1, 77])
    which = rng.choice(["forward", "dgrad", "wgrad", "int4"])
    gather = rng.random() < 0.5
    if which == "forward":
        check_forward(sizes, n, k, dtype, gather=gather, pad=pad, extra=extra, seed=seed)
    elif which == "dgrad":
        check_dgrad(sizes, n, k, dtype, pad=pad, extra=extra, seed=seed)
    elif which == "wgrad":
        check_wgrad(sizes, n, k, dtype, gather=gather, accumulate=rng.random() < 0.5, pad=pad,
                    extra=extra, seed=seed)
    else:
        group = rng.choice([32, 64, 128])
        k = group * rng.randint(1, max(1, widest // group))
        check_int4(sizes, rng.randint(1, widest), k, group, dtype,
                   scale_dtype=rng.choice([BF16, FP32]), zeros=rng.random() < 0.5, gather=gather,
                   pad=pad, seed=seed)


# ---------------------------------------------------------------------------
# the operations together, streams, graphs

def test_layer_with_the_finalize(cuda_lib):
    """Routing, both products and the finalize as a layer runs them, against
    float64 from the BF16 rows that each step stored."""
    T, K, E, H, inner = 45, 8, 12, 1024, 256
    ids = torch.stack([torch.randperm(E, generator=gen(t))[:K] for t in range(T)]).int()
    ids[3, 2] = ids[7] = -1
    tokens, rw = randn((T, H), 1), torch.rand((T, K), generator=gen(2)).cuda()
    up, down = weights(E, 2 * inner, H, 3), weights(E, H, inner, 4)
    norm = randn((H,), 5)
    off, idx, tok = mf.moe_expert_permutation(ids.cuda(), E)
    rows = T * K
    h = torch.zeros((rows, 2 * inner), dtype=BF16, device="cuda")
    mf.moe_grouped_gemm(tokens, up, off, h, row_index=tok)
    act = torch.nn.functional.silu(h[:, :inner].float()).mul(h[:, inner:]).to(BF16)
    y = torch.zeros((rows, H), dtype=BF16, device="cuda")
    mf.moe_grouped_gemm(act, down, off, y)
    out = torch.empty((T, H), dtype=BF16, device="cuda")
    mf.moe_finalize_rmsnorm(y, rw, idx, norm, out, eps=1e-5, gain_center=1.0,
                            weight_before_norm=False)
    # rows of the first product in float64, then of the second from the stored activations
    expert = torch.searchsorted(off[1:], torch.arange(rows, device="cuda").int(), right=True)
    live = int(off[-1])
    assert live == (ids >= 0).sum()
    for r in range(0, live, 17):
        a = tokens[tok[r]].double()
        we = up[expert[r]].double()
        within(h[r], we @ a, we.abs() @ a.abs(), H, BF16)
        b, wd = act[r].double(), down[expert[r]].double()
        within(y[r], wd @ b, wd.abs() @ b.abs(), inner, BF16)
    sums = (gathered(y, idx.flatten(), 0).view(T, K, H) * rw.double()[..., None]
            * (idx >= 0)[..., None]).sum(1)
    ref = sums / (sums.pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * (norm.double() + 1.0)
    # FP32 sums of 8 products and an FP32 norm of 1024 values before the BF16 round: the
    # norm's FP32 steps are within 2^-13 of the value (1024 additions), so is the sum
    mag = (gathered(y, idx.flatten(), 0).view(T, K, H).abs() * rw.double()[..., None]).sum(1)
    scale = 1 / (sums.pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * (norm.double() + 1.0).abs()
    tol = (2.0 ** -8 + 2.0 ** -12) * ref.abs() + 8 * 2.0 ** -23 * mag * scale + 1e-30
    assert ((out.double() - ref).abs() <= tol).all()
    assert (out[7] == 0).all()


def test_layer_with_4_bit_weights(cuda_lib):
    """One decoded token through 4-bit matrices into the finalize."""
    T, K, E, H = 1, 8, 16, 512
    ids = torch.randperm(E, generator=gen(1))[:K].int().view(T, K).cuda()
    x, rw = randn((T, H), 2), torch.rand((T, K), generator=gen(3)).cuda()
    q, s, z, w = int4_weights(E, H, H, 64, BF16, True, 4)
    off, idx, tok = mf.moe_expert_permutation(ids, E)
    y = torch.empty((T * K, H), dtype=BF16, device="cuda")
    mf.moe_grouped_gemv_int4(x, q, s, off, y, zeros=z, row_index=tok)
    for j in range(K):
        we = w[ids[0, j]]
        within(y[idx[0, j]], we @ x[0].double(), we.abs() @ x[0].double().abs(), H + 16, BF16)
    out = torch.empty((T, H), dtype=BF16, device="cuda")
    mf.moe_finalize_rmsnorm(y, rw, idx, torch.ones(H, dtype=BF16, device="cuda"), out, eps=1e-6,
                            gain_center=0.0, weight_before_norm=False)
    sums = (y[idx[0].long()].double() * rw[0].double()[:, None]).sum(0)
    ref = sums / (sums.pow(2).mean() + 1e-6).sqrt()
    mag = (y[idx[0].long()].double().abs() * rw[0].double()[:, None]).sum(0)
    tol = (2.0 ** -8 + 2.0 ** -12) * ref.abs() + \
        8 * 2.0 ** -23 * mag / (sums.pow(2).mean() + 1e-6).sqrt()
    assert ((out[0].double() - ref).abs() <= tol).all()


def training_step(tokens, w, ids, dy, E):
    """Loss = sum(y * dy) of one gathered product: gradients of tokens and weights."""
    off, idx, tok = mf.moe_expert_permutation(ids, E)
    rows, (n, k) = tok.numel(), w.shape[1:]
    y = torch.zeros((rows, n), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm(tokens, w, off, y, row_index=tok)
    dw = torch.empty(w.shape, dtype=FP32, device="cuda")
    mf.moe_grouped_gemm_wgrad(dy, tokens, off, dw, row_index=tok)
    d_rows = torch.empty((rows, k), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm_dgrad(dy, w, off, d_rows)
    dx = torch.empty(tokens.shape, dtype=FP32, device="cuda")
    mf.moe_permuted_row_sum(d_rows, idx, dx)
    return y, dx, dw, idx


def test_gradients_against_autograd_and_differences(cuda_lib):
    T, K, E, n, k = 40, 4, 6, 72, 136
    ids = torch.stack([torch.randperm(E, generator=gen(t))[:K] for t in range(T)]).int()
    ids[5, 1] = ids[9] = -1
    tokens, w, dy = randn((T, k), 1), randn((E, n, k), 2), randn((T * K, n), 3)
    y, dx, dw, idx = training_step(tokens, w, ids.cuda(), dy, E)
    tt, ww = tokens.double().requires_grad_(), w.double().requires_grad_()
    t_of, j_of = (ids >= 0).nonzero(as_tuple=True)
    rows = idx.cpu()[t_of, j_of].long()
    yy = torch.einsum("snk,sk->sn", ww[ids[t_of, j_of].long()], tt[t_of.cuda()])
    (yy * dy[rows.cuda()].double()).sum().backward()
    r = tokens.double().abs(), w.double().abs(), dy.double().abs()
    within(y[rows.cuda()], yy.detach(), torch.einsum(
        "snk,sk->sn", r[1][ids[t_of, j_of].long()], r[0][t_of.cuda()]), k, FP32)
    mag_w = torch.zeros_like(r[1]).index_add_(
        0, ids[t_of, j_of].long().cuda(),
        r[2][rows.cuda()][:, :, None] * r[0][t_of.cuda()][:, None, :])
    within(dw, ww.grad, mag_w, T, FP32)
    mag_x = torch.zeros_like(r[0]).index_add_(0, t_of.cuda(), torch.einsum(
        "snk,sn->sk", r[1][ids[t_of, j_of].long()], r[2][rows.cuda()]))
    # each row's gradient is itself rounded to FP32 once
    within(dx, tt.grad, mag_x, n + K + 1, FP32)
    assert (dx[9] == 0).all()
    # differences: the product is linear in each operand, so a step of one token's
    # value (a power of two) moves the loss by exactly step * gradient
    step = 2.0
    for t, c in ((0, 0), (5, 77), (39, 135)):
        moved = tokens.double().clone()
        moved[t, c] += step
        y2 = torch.einsum("snk,sk->sn", w.double()[ids[t_of, j_of].long()], moved[t_of.cuda()])
        diff = ((y2 - yy.detach()) * dy[rows.cuda()].double()).sum() / step
        assert abs(diff.item() - dx[t, c].item()) <= \
            (n + K + 1) * 2.0 ** -23 * mag_x[t, c].item() + 2.0 ** -24 * abs(diff.item()) + 1e-9


def all_ops(tokens, w, ids, dy, q, s, E):
    y, dx, dw, _ = training_step(tokens, w, ids, dy, E)
    off, _, tok = mf.moe_expert_permutation(ids, E)
    z = torch.zeros((tok.numel(), q.shape[1]), dtype=FP32, device="cuda")
    mf.moe_grouped_gemv_int4(tokens, q, s, off, z, row_index=tok)
    return y, dx, dw, z


def op_inputs(T=64, K=4, E=6, n=136, k=256):
    ids = torch.stack([torch.randperm(E, generator=gen(t))[:K] for t in range(T)]).int().cuda()
    q, s, _, _ = int4_weights(E, n, k, 64, BF16, False, 9)
    return randn((T, k), 1), randn((E, n, k), 2), ids, randn((T * K, n), 3), q, s, E


@pytest.mark.parametrize("programmatic", [True, False])
def test_bits_repeat_on_streams_and_in_graphs(cuda_lib, programmatic):
    args = op_inputs()
    mf.set_programmatic_launch(programmatic)
    try:
        want = all_ops(*args)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = all_ops(*args)
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        # two graphs of the same calls, replayed at once on two streams, on new inputs
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs = all_ops(*args)
            graphs.append((g, outs))
        args[0].mul_(-2)                       # exact in BF16 and FP32: results scale too
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            graphs[0][0].replay()
            with torch.cuda.stream(side):
                graphs[1][0].replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert torch.equal(outs[0], want[0] * -2)
            assert torch.equal(outs[1], want[1])
            assert torch.equal(outs[2], want[2] * -2)
            assert torch.equal(outs[3], want[3] * -2)
    finally:
        mf.set_programmatic_launch(True)


def test_decode_loop_in_a_graph(cuda_lib):
    """Decoded tokens one after the other: every launch right behind a finalize that lets
    its successor start early, with programmatic launch on and off."""
    T, K, E, H = 2, 8, 16, 4096
    q, s, z, _ = int4_weights(E, H, H, 128, BF16, True, 1)
    w = weights(E, H, H, 2)
    norm = torch.ones(H, dtype=BF16, device="cuda")
    rw = torch.rand((T, K), generator=gen(3)).cuda()
    ids = torch.stack([torch.randperm(E, generator=gen(t))[:K] for t in range(T)]).int().cuda()
    start = randn((T, H), 4)

    def steps():
        h, kept = start, []
        for i in range(4):
            step_ids = ((ids + i) % E).contiguous()
            off, idx, tok = mf.moe_expert_permutation(step_ids, E)
            y = torch.empty((T * K, H), dtype=BF16, device="cuda")
            if i % 2:
                mf.moe_grouped_gemv_int4(h, q, s, off, y, zeros=z, row_index=tok)
            else:
                mf.moe_grouped_gemm(h, w, off, y, row_index=tok)
            h = torch.empty((T, H), dtype=BF16, device="cuda")
            mf.moe_finalize_rmsnorm(y, rw, idx, norm, h, eps=1e-6, gain_center=0.0,
                                    weight_before_norm=False)
            kept.append(h)
        return kept

    results = []
    try:
        for programmatic in (True, False):
            mf.set_programmatic_launch(programmatic)
            results.append([t.clone() for t in steps()])
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs = steps()
            for _ in range(3):
                g.replay()
            torch.cuda.synchronize()
            results.append(outs)
    finally:
        mf.set_programmatic_launch(True)
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)
    assert all(torch.isfinite(t).all() for t in results[0])


def test_two_streams_at_once(cuda_lib):
    """Large products on two streams at the same time give what each gives alone."""
    jobs = []
    for seed in (1, 2):
        sizes = [700, 0, 300, 90 * seed]
        x, w = padded(sum(sizes), 1032, seed, 0), weights(4, 1416, 1032, seed + 5)
        q, s, z, _ = int4_weights(4, 1000, 1024, 64, BF16, True, seed)
        jobs.append((x, w, offsets_of(sizes), q, s, z, padded(sum(sizes), 1024, seed + 9, 0)))

    def run(job, outs=None):
        x, w, off, q, s, z, x4 = job
        outs = outs or (torch.empty((x.shape[0], 1416), dtype=BF16, device="cuda"),
                        torch.empty((x.shape[0], 1000), dtype=FP32, device="cuda"),
                        torch.empty(w.shape, dtype=FP32, device="cuda"))
        mf.moe_grouped_gemm(x, w, off, outs[0])
        mf.moe_grouped_gemv_int4(x4, q, s, off, outs[1], zeros=z)
        mf.moe_grouped_gemm_wgrad(outs[0], x, off, outs[2])
        return outs

    alone = [run(j) for j in jobs]
    torch.cuda.synchronize()
    together = [tuple(torch.empty_like(t) for t in a) for a in alone]
    streams = [torch.cuda.Stream() for _ in jobs]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for st, job, outs in zip(streams, jobs, together):
            with torch.cuda.stream(st):
                run(job, outs)
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_stream_argument(cuda_lib):
    """Every call on a stream that is not the current one, outputs allocated there."""
    T, K, E, n, k = 33, 4, 6, 72, 128
    ids = torch.randint(0, E, (T, K), generator=gen(1), dtype=torch.int32).cuda()
    tokens, w = randn((T, k), 2), randn((E, n, k), 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    off, idx, tok = mf.moe_expert_permutation(ids, E, stream=side)
    y = torch.empty((T * K, n), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm(tokens, w, off, y, row_index=tok, stream=side)
    side.synchronize()
    off2, idx2, tok2 = mf.moe_expert_permutation(ids, E)
    y2 = torch.empty_like(y)
    mf.moe_grouped_gemm(tokens, w, off2, y2, row_index=tok2)
    torch.cuda.synchronize()
    for a, b in ((off, off2), (idx, idx2), (tok, tok2), (y, y2)):
        assert torch.equal(a, b)


def test_far_rows(cuda_lib):
    """Element offsets past 2^31: the last rows of a buffer of more than 4 GB."""
    rows, k, n = 270000, 8192, 64
    x = torch.zeros((rows, k), dtype=BF16, device="cuda")
    x[-300:] = randn((300, k), 1)
    w = weights(2, n, k, 2)
    off = torch.tensor([0, rows - 200, rows], dtype=torch.int32, device="cuda")
    index = torch.arange(rows, dtype=torch.int32, device="cuda")
    last = x[-300:].double()
    for ix in (None, index):
        out = torch.empty((rows, n), dtype=FP32, device="cuda")
        mf.moe_grouped_gemm(x, w, off, out, row_index=ix)
        for e, sl in ((0, slice(0, 100)), (1, slice(100, 300))):
            within(out[-300:][sl], last[sl] @ w[e].double().t(),
                   last[sl].abs() @ w[e].double().abs().t(), k, FP32)
        assert (out[:-300] == 0).all()
    dx = torch.empty((rows, k), dtype=BF16, device="cuda")
    mf.moe_grouped_gemm_dgrad(torch.zeros((rows, n), dtype=BF16, device="cuda"), w, off, dx)
    assert (dx == 0).all()
    idx = torch.tensor([[rows - 1, 0], [rows - 300, rows - 299]], dtype=torch.int32, device="cuda")
    s = torch.empty((2, k), dtype=FP32, device="cuda")
    mf.moe_permuted_row_sum(x, idx, s)
    assert torch.equal(s, x[idx.long()].float().sum(1))
