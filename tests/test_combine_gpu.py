"""moe_dispatch, moe_combine and moe_combine_backward against float64 (and, where one
rounding of an FP32 product is all there is, bit for bit)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
U = 2.0 ** -24  # half a step of FP32


def make(T, K, H, rows_dtype=BF16, token_dtype=BF16, weights="fp32", dropped=0.1, extra=3, seed=0,
         pad=0):
    """A map with distinct rows, `dropped` slots and `extra` rows that no slot names; rows
    that no slot names and the padding behind the columns hold NaN."""
    g = torch.Generator().manual_seed(seed)
    n = T * K
    rows = n + extra
    idx = torch.randperm(rows, generator=g)[:n].int()
    drop = torch.rand(n, generator=g) < dropped
    bad = torch.tensor([-1, rows, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 4, (n,), generator=g)]
    idx = torch.where(drop, bad.int(), idx).view(T, K)
    live = (idx >= 0) & (idx < rows)
    w = torch.randn((T, K), generator=g)
    # weights of slots without a row have no effect
    w = torch.where(live, w, torch.tensor(float("nan")))
    if weights == "bf16":
        w = w.bfloat16()
    elif weights == "packed":
        bits = w.bfloat16().view(torch.int16).int() & 0xFFFF
        w = (torch.randint(-2 ** 15, 2 ** 15, (T, K), generator=g).int() << 16) | bits

    def buffer(m, dtype, fill=None):
        b = torch.full((m, H + pad), float("nan"), dtype=dtype)
        if fill is not None:
            b[:, :H] = fill
        return b.cuda()[:, :H]

    named = torch.zeros(rows, dtype=torch.bool)
    named[idx[live].long()] = True
    p = torch.randn((rows, H), generator=g)
    p[~named] = float("nan")
    s = dict(T=T, K=K, H=H, rows=rows, idx=idx.cuda(), live=live.cuda(), w=w.cuda(),
             named=named.cuda(), p=buffer(rows, rows_dtype, p),
             x=buffer(T, token_dtype, torch.randn((T, H), generator=g)),
             out_rows=buffer(rows, rows_dtype), out_tokens=buffer(T, token_dtype))
    if weights == "packed":
        s["wf"] = (s["w"] << 16).view(FP32)
    else:
        s["wf"] = s["w"].float()
    s["wf"] = torch.where(s["live"], s["wf"], torch.zeros_like(s["wf"]))
    s["rows_of"] = torch.where(s["live"], s["idx"], torch.zeros_like(s["idx"])).long()
    return s


def gathered(s):
    """The slots' rows in float64, zeros where there is none."""
    r = s["p"][s["rows_of"]].double()
    return torch.where(s["live"].unsqueeze(-1), r, torch.zeros_like(r))


def check_dispatch(s, out, weighted=True):
    v = s["x"].float().unsqueeze(1).expand(s["T"], s["K"], s["H"])
    if weighted:
        v = v * s["wf"].unsqueeze(-1)
    want = v.to(out.dtype)
    assert torch.equal(out[s["idx"][s["live"]].long()], want[s["live"]])
    assert out[~s["named"]].isnan().all()   # left as they were


def check_combine(s, out):
    terms = gathered(s) * s["wf"].double().unsqueeze(-1)
    want = terms.sum(1)
    # K multiply-adds, each off by half a step of a partial sum, and the result's rounding
    bound = s["K"] * U * terms.abs().sum(1) * (1 + 2 ** -10)
    bound = bound + (want.abs() + bound) * (torch.finfo(out.dtype).eps / 2)
    assert ((out.double() - want).abs() <= bound).all()


def check_grad_weights(s, gw):
    terms = gathered(s) * s["x"].double().unsqueeze(1)
    want = terms.sum(-1)
    # additions on the longest way: a chunk's 4, the two chains' one, a thread's chunks (of four
    # columns or more; a team has 32 threads at least), 5 between lanes, up to 16 warps; a
    # product's own half step
    depth = 1 + 4 + 1 + -(-s["H"] // 128) + 5 + 16
    bound = depth * U * terms.abs().sum(-1) * (1 + 2 ** -10)
    bound = bound + (want.abs() + bound) * (torch.finfo(gw.dtype).eps / 2)
    assert ((gw.double() - want).abs() <= bound).all()
    assert (gw[~s["live"]] == 0).all()


SIZES = [(1, 1, 8), (1, 8, 4096), (3, 2, 16), (5, 32, 264), (2, 5, 520), (17, 6, 2056),
         (129, 3, 256), (130, 9, 512), (700, 8, 1032), (1300, 4, 2872), (40, 8, 7168),
         (2, 1, 65544)]


@pytest.mark.parametrize("T,K,H", SIZES)
@pytest.mark.parametrize("rows_dtype", [BF16, FP32])
@pytest.mark.parametrize("token_dtype", [BF16, FP32])
def test_parity(cuda_lib, T, K, H, rows_dtype, token_dtype):
    mf = cuda_lib
    for i, (weights, pad) in enumerate((("fp32", 0), ("bf16", 8), ("packed", 24))):
        s = make(T, K, H, rows_dtype, token_dtype, weights, seed=i, pad=pad)
        assert mf.moe_dispatch(s["x"], s["idx"], s["out_rows"],
                               expert_weights=s["w"]) is s["out_rows"]
        check_dispatch(s, s["out_rows"])
        s["out_rows"].fill_(float("nan"))
        mf.moe_dispatch(s["x"], s["idx"], s["out_rows"])
        check_dispatch(s, s["out_rows"], weighted=False)
        assert mf.moe_combine(s["p"], s["w"], s["idx"], s["out_tokens"]) is s["out_tokens"]
        check_combine(s, s["out_tokens"])
        for gw_dtype in (FP32, BF16):
            s["out_rows"].fill_(float("nan"))
            gw = torch.full((T, K), float("nan"), dtype=gw_dtype, device="cuda")
            mf.moe_combine_backward(s["x"], s["p"], s["w"], s["idx"], s["out_rows"], gw)
            check_dispatch(s, s["out_rows"])
            check_grad_weights(s, gw)
        alone = torch.full((T, K), float("nan"), dtype=FP32, device="cuda")
        mf.moe_combine_backward(s["x"], s["p"], None, s["idx"], None, alone)
        both = torch.empty_like(alone)
        mf.moe_combine_backward(s["x"], s["p"], s["w"], s["idx"], s["out_rows"], both)
        assert torch.equal(alone, both)
        s["out_rows"].fill_(float("nan"))
        mf.moe_combine_backward(s["x"], None, s["w"], s["idx"], s["out_rows"], None)
        check_dispatch(s, s["out_rows"])
        if pad:   # the columns behind the rows are not touched
            for name in ("out_rows", "out_tokens"):
                t = s[name]
                whole = t.as_strided((t.shape[0], H + pad), (H + pad, 1))
                assert whole[:, H:].isnan().all()


@pytest.mark.parametrize("T", [1, 2, 152, 153, 608, 4001])
@pytest.mark.parametrize("H", [1528, 1536, 1544, 2048, 2056])
@pytest.mark.parametrize("K", [3, 4, 5, 9])
def test_team_edges(cuda_lib, T, H, K):
    """Around the choices of how many threads take a token's gradients, and how many slots."""
    s = make(T, K, H, seed=T)
    gw = torch.full((T, K), float("nan"), device="cuda")
    cuda_lib.moe_combine_backward(s["x"], s["p"], s["w"], s["idx"], s["out_rows"], gw)
    check_dispatch(s, s["out_rows"])
    check_grad_weights(s, gw)


def test_a_row_for_several_slots(cuda_lib):
    """Combining may read a row more than once, for the weights' gradient too."""
    s = make(9, 8, 264)
    s["idx"][:, :] = 5
    s["idx"][2, 3] = -1
    s["live"] = s["idx"] >= 0
    s["rows_of"] = s["idx"].clamp(min=0).long()
    s["p"][5] = 0.5
    w = torch.randn((9, 8), device="cuda")
    s["wf"] = torch.where(s["live"], w, torch.zeros_like(w))
    cuda_lib.moe_combine(s["p"], w, s["idx"], s["out_tokens"])
    check_combine(s, s["out_tokens"])
    gw = torch.empty((9, 8), device="cuda")
    cuda_lib.moe_combine_backward(s["x"], s["p"], None, s["idx"], None, gw)
    check_grad_weights(s, gw)


def test_no_rows_and_no_tokens(cuda_lib):
    mf = cuda_lib
    idx = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    idx[0, 0] = 0   # outside: there are no rows
    w = torch.full((4, 2), float("nan"), device="cuda")
    none = torch.empty((0, 64), dtype=BF16, device="cuda")
    x = torch.randn((4, 64), device="cuda").bfloat16()
    out = torch.full((4, 64), float("nan"), dtype=BF16, device="cuda")
    mf.moe_dispatch(x, idx, none)
    mf.moe_combine(none, w, idx, out)
    assert (out == 0).all()
    gw = torch.full((4, 2), float("nan"), device="cuda")
    mf.moe_combine_backward(x, none, w, idx, none.clone(), gw)
    assert (gw == 0).all()
    e = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    rows = torch.ones((3, 64), dtype=BF16, device="cuda")
    mf.moe_dispatch(none, e, rows)
    mf.moe_combine(rows, e.float(), e, none)
    mf.moe_combine_backward(none, rows, e.float(), e, rows.clone(), e.float())
    assert (rows == 1).all()


def test_infinities_and_nan(cuda_lib):
    mf = cuda_lib
    inf, nan = float("inf"), float("nan")
    p = torch.tensor([1.0, inf, -inf, nan], device="cuda").unsqueeze(1).expand(4, 16).contiguous()
    idx = torch.tensor([[0, 1], [1, 2], [0, 3], [0, -1], [1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 1.0], [1, 1], [1, 1], [2, nan], [0, inf]], device="cuda")
    out = torch.empty((5, 16), device="cuda")
    mf.moe_combine(p, w, idx, out)
    want = torch.tensor([inf, nan, nan, 2.0, nan], device="cuda")
    assert torch.equal(out[:, 0].nan_to_num(7.0, posinf=9.0), want.nan_to_num(7.0, posinf=9.0))
    gw = torch.empty((5, 2), device="cuda")
    dy = torch.ones((5, 16), device="cuda")
    mf.moe_combine_backward(dy, p, w, idx, None, gw)
    want = torch.tensor([[16, inf], [inf, -inf], [16, nan], [16, 0], [inf, 0]], device="cuda")
    assert torch.equal(gw.isnan(), want.isnan())
    assert torch.equal(gw.nan_to_num(7.0), want.nan_to_num(7.0))


def test_against_differences(cuda_lib):
    """The gradients against difference quotients of the forward pass, which is linear in the
    rows and in the weights."""
    mf = cuda_lib
    s = make(37, 5, 136, FP32, FP32, dropped=0.2, seed=4)
    s["p"].nan_to_num_(0.0)
    w = s["w"].nan_to_num(0.0)
    dy = s["x"]
    gp = torch.zeros((s["rows"], s["H"]), device="cuda")
    gw = torch.zeros_like(w)
    mf.moe_combine_backward(dy, s["p"], w, s["idx"], gp, gw)

    def loss(p, wt):
        out = torch.empty((s["T"], s["H"]), device="cuda")
        mf.moe_combine(p, wt, s["idx"], out)
        return (out.double() * dy.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(1)
    for grad, at in ((gp, "p"), (gw, "w")):
        d = torch.randn(grad.shape, generator=g, device="cuda")
        h = 0.5
        if at == "p":
            got = (loss(s["p"] + h * d, w) - loss(s["p"] - h * d, w)) / (2 * h)
        else:
            got = (loss(s["p"], w + h * d) - loss(s["p"], w - h * d)) / (2 * h)
        want = (grad.double() * d.double()).sum()
        # each loss: K + 3 roundings of FP32 in every column, over terms of this size
        size = (gathered(s).abs() * w.double().abs().unsqueeze(-1) + 4).sum(1).mul(dy.double().abs())
        assert (got - want).abs() <= 2 * 8 * 2 * U * size.sum() * 4


def test_chain_as_used(cuda_lib):
    """Permutation, rows in, one product, rows out and all gradients, against float64."""
    mf = cuda_lib
    T, K, E, H, N = 200, 4, 6, 264, 136
    g = torch.Generator().manual_seed(3)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int()
    ids[5, 1] = -1
    ids[9] = -1
    ids = ids.cuda()
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    w = torch.rand((T, K), generator=g).cuda()
    weight = (torch.randn((E, N, H), generator=g) * H ** -0.5).bfloat16().cuda()
    off, idx, tok = mf.moe_expert_permutation(ids, E)
    n = int(off[E])
    rows = torch.full((T * K, H), float("nan"), dtype=BF16, device="cuda")
    mf.moe_dispatch(x, idx, rows)
    assert torch.equal(rows[:n], x[tok[:n].long()]) and rows[n:].isnan().all()
    y = torch.full((T * K, N), float("nan"), dtype=FP32, device="cuda")
    mf.moe_grouped_gemm(rows, weight, off, y)
    out = torch.empty((T, N), device="cuda")
    mf.moe_combine(y, w, idx, out)
    live = (ids >= 0)
    yy = torch.einsum("th,tknh->tkn", x.double(), weight.double()[ids.clamp(min=0).long()])
    yy = yy * live.unsqueeze(-1)
    want = (yy * w.double().unsqueeze(-1)).sum(1)
    assert (out.double() - want).norm() <= 2e-6 * want.norm()
    dy = torch.randn((T, N), generator=g).cuda()
    d_y = torch.full_like(y, float("nan"))
    d_w = torch.empty((T, K), device="cuda")
    mf.moe_combine_backward(dy, y, w, idx, d_y, d_w)
    want_w = (yy * dy.double().unsqueeze(1)).sum(-1)
    assert (d_w.double() - want_w).norm() <= 2e-6 * want_w.norm()
    want_y = (dy.unsqueeze(1) * w.unsqueeze(-1))
    assert torch.equal(d_y[idx[live].long()], want_y[live])
    d_rows = torch.empty((T * K, H), dtype=FP32, device="cuda")
    d_yb = d_y.bfloat16()
    mf.moe_grouped_gemm_dgrad(d_yb, weight, off, d_rows)
    d_x = torch.empty((T, H), device="cuda")
    mf.moe_permuted_row_sum(d_rows, idx, d_x)
    slot = torch.where(live, idx, torch.zeros_like(idx)).long()
    want_x = torch.einsum("tkn,tknh->th", (d_yb[slot].double() * live.unsqueeze(-1)).nan_to_num(0),
                          weight.double()[ids.clamp(min=0).long()])
    assert (d_x.double() - want_x).norm() <= 2e-6 * want_x.norm()


def test_weighted_way_in_and_its_gradients(cuda_lib):
    """out[m] = w x: the gradient of x by moe_combine, of w by moe_combine_backward."""
    mf = cuda_lib
    s = make(50, 4, 264, FP32, FP32, seed=8)
    d_out = s["p"]
    d_x = torch.empty((50, 264), device="cuda")
    mf.moe_combine(d_out, s["w"], s["idx"], d_x)
    check_combine(s, d_x)
    d_w = torch.empty((50, 4), device="cuda")
    mf.moe_combine_backward(s["x"], d_out, None, s["idx"], None, d_w)
    check_grad_weights(s, d_w)


def test_streams_and_graph(cuda_lib):
    """Two streams at once, and a captured pass replayed with other inputs."""
    mf = cuda_lib
    a, b = make(300, 8, 1032, seed=1), make(300, 8, 1032, seed=2)
    gwa, gwb = (torch.empty((300, 8), device="cuda") for _ in range(2))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, gw, st in ((a, gwa, streams[0]), (b, gwb, streams[1])):
            mf.moe_combine(s["p"], s["w"], s["idx"], s["out_tokens"], stream=st)
            mf.moe_combine_backward(s["x"], s["p"], s["w"], s["idx"], s["out_rows"], gw, stream=st)
    torch.cuda.synchronize()
    for s, gw in ((a, gwa), (b, gwb)):
        check_combine(s, s["out_tokens"])
        check_dispatch(s, s["out_rows"])
        check_grad_weights(s, gw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mf.moe_dispatch(a["x"], a["idx"], a["out_rows"], expert_weights=a["w"])
        mf.moe_combine_backward(a["x"], a["p"], None, a["idx"], None, gwa)
        mf.moe_combine(a["p"], a["w"], a["idx"], a["out_tokens"])
    for name in ("x", "idx", "w", "p", "live", "named", "rows_of", "wf"):
        a[name].copy_(b[name])
    a["out_rows"].fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    check_dispatch(a, a["out_rows"])
    check_grad_weights(a, gwa)
    check_combine(a, a["out_tokens"])


def test_repeats_bit_for_bit(cuda_lib):
    s = make(900, 8, 2056, seed=6)
    runs = []
    for _ in range(3):
        gw = torch.empty((900, 8), device="cuda")
        out = torch.empty((900, 2056), dtype=BF16, device="cuda")
        cuda_lib.moe_combine_backward(s["x"], s["p"], s["w"], s["idx"], s["out_rows"], gw)
        cuda_lib.moe_combine(s["p"], s["w"], s["idx"], out)
        runs.append((gw, out))
    for gw, out in runs[1:]:
        assert torch.equal(gw, runs[0][0]) and torch.equal(out, runs[0][1])


def test_offsets_beyond_32_bits(cuda_lib):
    """Rows whose elements begin behind 2^32 (a wide stride)."""
    mf = cuda_lib
    rows, H, ld = 70, 64, 2 ** 26
    big = torch.empty(rows * ld, dtype=BF16, device="cuda").view(rows, ld)[:, :H]
    s = make(16, 4, H, extra=rows - 64, seed=9)
    mf.moe_dispatch(s["x"], s["idx"], big, expert_weights=s["w"])
    slots = s["idx"][s["live"]].long()
    want = (s["x"].float().unsqueeze(1) * s["wf"].unsqueeze(-1)).bfloat16()
    assert int(slots.max()) * ld > 2 ** 31
    assert torch.equal(big[slots], want[s["live"]])
    big.copy_(s["p"])
    mf.moe_combine(big, s["w"], s["idx"], s["out_tokens"])
    check_combine(s, s["out_tokens"])
    gw = torch.empty((16, 4), device="cuda")
    mf.moe_combine_backward(s["x"], big, None, s["idx"], None, gw)
    check_grad_weights(s, gw)


def test_one_wide_row(cuda_lib):
    """A single row of more columns than the tokens', not a multiple of 8."""
    rows = torch.randn((1, 76), device="cuda").bfloat16()
    idx = torch.tensor([[0, -1], [1, 0]], dtype=torch.int32, device="cuda")
    w = torch.rand((2, 2), device="cuda")
    out = torch.empty((2, 64), device="cuda")
    cuda_lib.moe_combine(rows, w, idx, out)
    assert torch.equal(out, torch.stack([w[0, 0], w[1, 1]]).unsqueeze(1) * rows[:, :64].float())
