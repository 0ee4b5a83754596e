"""The 4-bit floating point operations against float64: quantisation bit for bit, the
products within the bounds of their additions."""
import pytest
import torch

import fp4_common as fp4

pytestmark = pytest.mark.gpu

BF16, FP32, U8 = torch.bfloat16, torch.float32, torch.uint8
MX, NV = fp4.MX, fp4.NV
U = 2.0 ** -24  # half a step of FP32
NAN = float("nan")


def buffers(shape, k, fmt, pad=0):
    """Packed values and scales with 0xA5 in and behind the rows (`pad` further 16 bytes)."""
    g = k // fp4.BLOCK[fmt]
    q = torch.full((*shape, k // 2 + 16 * pad), 0xA5, dtype=U8, device="cuda")
    s = torch.full((*shape, -(-g // 16) * 16 + 16 * pad), 0xA5, dtype=U8, device="cuda")
    return q[..., :k // 2], s[..., :g].view(fmt)


def untouched(t):
    """The bytes behind the rows."""
    rows = t.stride(-2)
    whole = t.view(U8).as_strided((t.shape[0], rows), (rows, 1))
    return bool((whole[:, t.shape[1]:] == 0xA5).all())


def check_quantized(mf, x, fmt, factor=None, pad=0):
    q, s = buffers((x.shape[0],), x.shape[1], fmt, pad)
    got = mf.moe_quantize_fp4(x, q, s, factor=factor)
    assert got[0] is q and got[1] is s
    codes, byte = fp4.quantize(x, fmt, factor)
    assert torch.equal(s.view(U8), byte)
    assert torch.equal(q, fp4.pack(codes))
    assert untouched(q) and untouched(s)
    return q, s


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 4096), (3, 96), (7, 2880), (130, 160), (33, 4160),
                                    (513, 32), (2, 65568), (300, 1024)])
def test_quantize(cuda_lib, fmt, dtype, rows, k):
    g = torch.Generator(device="cuda").manual_seed(rows * k)
    wide = torch.randn((rows, k + 24), generator=g, device="cuda")
    wide *= torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g, device="cuda").float())
    wide[:, 5::64] *= 8
    wide[rows // 2, :k // 2] = 0
    wide = wide.to(dtype)
    for x, pad in ((wide[:, :k].contiguous(), 0), (wide[:, 8:k + 8], 1)):
        check_quantized(cuda_lib, x, fmt, pad=pad)
        for f in (1.0, 0.37, 2688.0):
            check_quantized(cuda_lib, x, fmt, torch.tensor([f], device="cuda"))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_quantize_borders(cuda_lib, fmt, dtype):
    """Values on the borders between neighbouring codes and next to them, for every scale of a
    binade and scales far out."""
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    rows = []
    for e in (-100, -9, -6, 0, 1, 8, 100):
        for m in range(8, 16):
            scale = m / 8 * 2.0 ** e if fmt == NV else 2.0 ** e
            v = torch.zeros(32, dtype=torch.float64)
            v[0] = v[16] = 6 * scale
            for i, b in enumerate(borders):
                t = (b * scale).to(dtype)
                step = torch.finfo(dtype).eps
                v[1 + 2 * i] = t.double()
                v[2 + 2 * i] = -(t.double() * (1 + step)).to(dtype).double()
                v[17 + 2 * i] = -t.double()
                v[18 + 2 * i] = (t.double() * (1 - step)).to(dtype).double()
            rows.append(v)
    x = torch.stack(rows).to(dtype).cuda()
    q, s = check_quantized(cuda_lib, x, fmt)
    got = fp4.values(q, s)[:, 1:15:2]
    inside = (got[:, 0] != 0) | (got[:, 1] != 0)   # not the scales that underflow or saturate
    ties = torch.tensor([0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0], dtype=torch.float64, device="cuda")
    scale = fp4.scale_values(s)[:, :1]
    if fmt == MX:
        assert torch.equal(got, ties * scale)
    else:
        mid = (scale[:, 0] > 0.02) & (scale[:, 0] < 448) & inside
        assert mid.sum() >= 24 and torch.equal(got[mid], (ties * scale)[mid])


@pytest.mark.parametrize("fmt", [MX, NV])
def test_quantize_every_bf16(cuda_lib, fmt):
    """Every BF16 value in a block whose largest is 6 or itself, and alone."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    v = bits.view(BF16)
    x = torch.zeros((65536, 64), dtype=BF16, device="cuda")
    x[:, 3] = v
    x[:, 17] = 6.0
    x[:, 16:32] = torch.where(x[:, 16:32] == 0, v.unsqueeze(1), x[:, 16:32])
    x[:, 40] = v
    check_quantized(cuda_lib, x, fmt)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_quantize_scale_ties(cuda_lib, fmt):
    """Largest magnitudes that put the scale on a border of its format, and next to it."""
    m = torch.arange(17, 32, 2, dtype=torch.float64) / 16   # midpoints of E4M3's neighbours
    e = torch.arange(-9, 9, dtype=torch.float64)
    mid = (m.unsqueeze(1) * torch.exp2(e)).flatten() * 6
    near = torch.cat((mid, torch.nextafter(mid.float(), torch.tensor(1e30)).double(),
                      torch.nextafter(mid.float(), torch.tensor(0.0)).double(),
                      torch.exp2(e), torch.nextafter(torch.exp2(e).float(), torch.tensor(0.0)).double(),
                      torch.tensor([448.0 * 6, 464 * 6, 480 * 6, 3e38, 2.0 ** -9 * 6, 2.0 ** -10 * 6,
                                    2.0 ** -149, 2.0 ** -126, 2.0 ** -127, 1e-40])))
    x = torch.zeros((near.numel(), 32), dtype=FP32)
    x[:, 7] = near.float()
    x[:, 21] = -near.float()
    x[:, 8] = near.float() * 0.3
    check_quantized(cuda_lib, x.cuda(), fmt)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_quantize_what_is_not_finite(cuda_lib, fmt, dtype):
    x = torch.randn((6, 96), device="cuda").to(dtype)
    x[0, 5] = float("inf")
    x[1, 40] = -float("inf")
    x[2, 95] = NAN
    x[3, :] = -0.0
    x[4, 3], x[4, 70] = NAN, float("inf")
    q, s = check_quantized(cuda_lib, x, fmt)
    v = fp4.values(q, s)
    assert v[0, :16].isnan().all() and not v[0, 32:].isnan().any()
    # an overflow by the factor is an infinity
    check_quantized(cuda_lib, torch.full((1, 32), 1e30, device="cuda"), fmt,
                    torch.tensor([1e30], device="cuda"))


@pytest.mark.parametrize("fmt", [MX, NV])
def test_dequantize_every_code(cuda_lib, fmt):
    """All 16 codes with all 256 scales."""
    k = 32
    q, s = buffers((256,), k, fmt)
    codes = (torch.arange(k, device="cuda") % 16).to(U8).expand(256, k)
    q.copy_(fp4.pack(codes))
    s.view(U8).copy_(torch.arange(256, dtype=U8, device="cuda").unsqueeze(1).expand(256, s.shape[1]))
    want = fp4.values(q, s)
    for dtype in (FP32, BF16):
        out = torch.zeros((256, k + 8), dtype=dtype, device="cuda")[:, :k]
        assert cuda_lib.moe_dequantize_fp4(q, s, out) is out
        w = want.float().to(dtype)
        assert torch.equal(out.isnan(), w.isnan())
        assert torch.equal(out.nan_to_num(1.0, posinf=7.0, neginf=-7.0),
                           w.nan_to_num(1.0, posinf=7.0, neginf=-7.0))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,k", [(1, 32), (5, 96), (129, 2880), (700, 512)])
def test_dequantize(cuda_lib, fmt, rows, k):
    g = torch.Generator(device="cuda").manual_seed(k)
    q, s = buffers((rows,), k, fmt, pad=1)
    q.copy_(torch.randint(0, 256, q.shape, generator=g, device="cuda", dtype=U8))
    s.view(U8).copy_(torch.randint(100, 126, s.shape, generator=g, device="cuda", dtype=U8))
    for dtype in (FP32, BF16):
        out = torch.full((rows, k + 16), NAN, dtype=dtype, device="cuda")
        cuda_lib.moe_dequantize_fp4(q, s, out[:, :k])
        assert torch.equal(out[:, :k].double(), fp4.values(q, s))
        assert out[:, k:].isnan().all()


@pytest.mark.parametrize("fmt", [MX, NV])
def test_there_and_back_on_streams_and_in_a_graph(cuda_lib, fmt):
    """Two streams at once with buffers of their own, and a replay with other rows."""
    rows, k = 133, 1056
    x = torch.randn((rows, k), device="cuda").bfloat16()
    factor = torch.full((1,), 0.75, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for st in streams * 2:
        q = cuda_lib.moe_fp4_empty((rows,), k, fmt, stream=st)
        with torch.cuda.stream(st):
            out = torch.empty((rows, k), device="cuda")
        cuda_lib.moe_quantize_fp4(x, *q, factor=factor, stream=st)
        cuda_lib.moe_dequantize_fp4(*q, out, stream=st)
        got.append((q, out))
    torch.cuda.synchronize()
    codes, byte = fp4.quantize(x, fmt, factor)
    for q, out in got:
        assert torch.equal(q[0], fp4.pack(codes)) and torch.equal(q[1].view(U8), byte)
        assert torch.equal(out.double(), fp4.values(*q))
    q, out = got[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.moe_quantize_fp4(x, *q, factor=factor)
        cuda_lib.moe_dequantize_fp4(*q, out)
    x.copy_(torch.randn((rows, k), device="cuda"))
    factor.fill_(-3.0)
    graph.replay()
    torch.cuda.synchronize()
    codes, byte = fp4.quantize(x, fmt, factor)
    assert torch.equal(q[0], fp4.pack(codes)) and torch.equal(q[1].view(U8), byte)
    assert torch.equal(out.double(), fp4.values(*q))


# ---------------------------------------------------------------------------
# the product

def layer(sizes, n, k, fmt, *, gather=False, x_rows=None, extra=0, seed=0, pad=0, factor=False,
          scale_range=None):
    """Operands of a product with `sizes` rows an expert; `extra` rows behind the last."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, rows = len(sizes), sum(sizes) + extra
    off = torch.tensor([0] + sizes).cumsum(0).int().cuda()
    x_rows = x_rows or (max(1, rows // 3) if gather else max(rows, 1))
    lo, hi = scale_range or ((120, 134) if fmt == MX else (0x20, 0x58))

    def random(shape):
        q, s = buffers(shape, k, fmt, pad)
        q.copy_(torch.randint(0, 256, q.shape, generator=g, device="cuda", dtype=U8))
        s.view(U8).copy_(torch.randint(lo, hi, s.shape, generator=g, device="cuda", dtype=U8))
        return q, s

    s = dict(sizes=sizes, off=off, rows=rows, n=n, k=k, fmt=fmt, E=E)
    s["x"], s["xs"] = random((x_rows,))
    s["w"], s["ws"] = random((E, n))
    s["index"] = None
    if gather:
        s["index"] = torch.randint(0, x_rows, (rows,), generator=g, device="cuda").int()
        bad = torch.rand(rows, generator=g, device="cuda") < 0.1
        s["index"][bad] = torch.tensor([-1, x_rows, 2 ** 31 - 1, -2 ** 31], device="cuda").int()[
            torch.randint(0, 4, (int(bad.sum()),), generator=g, device="cuda")]
    s["factor"] = torch.randn(E, generator=g, device="cuda") if factor else None
    return s


def product(mf, s, dtype, ld=None):
    out = torch.full((s["rows"], ld or s["n"]), NAN, dtype=dtype, device="cuda")
    got = mf.moe_grouped_gemm_fp4(s["x"], s["xs"], s["w"], s["ws"], s["off"], out[:, :s["n"]],
                                  row_index=s["index"], factor=s["factor"])
    assert got.data_ptr() == out.data_ptr()
    return out


def exact(s):
    """The product in float64, and the sums of its terms' magnitudes."""
    x = fp4.values(s["x"], s["xs"])
    if s["index"] is not None:
        i = s["index"].long()
        fine = (i >= 0) & (i < x.shape[0])
        x = x[i.clamp(0, x.shape[0] - 1)] * fine.unsqueeze(1)
    y = torch.zeros((s["rows"], s["n"]), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    at = 0
    for e, m in enumerate(s["sizes"]):
        w = fp4.values(s["w"][e], s["ws"][e])
        f = 1.0 if s["factor"] is None else s["factor"][e].double()
        y[at:at + m] = x[at:at + m] @ w.t() * f
        size[at:at + m] = x[at:at + m].abs() @ w.abs().t() * abs(f)
        at += m
    return y, size


def check(s, out):
    n, live = s["n"], sum(s["sizes"])
    want, size = exact(s)
    want, size, got = want[:live], size[:live], out[:live, :n].double()
    # one accumulator in the tensor cores, which truncate a partial sum every 64 values (by 2^-22
    # of the terms at most); FP32 results, and longer sums than 131072, leave them every 40
    # truncations, and the pieces are added in FP32, by up to 16 warps; the factor's product
    cuts, adds = -(-s["k"] // 64), -(-s["k"] // 32) + 16
    if out.dtype == FP32 or s["k"] > 131072:
        cuts = min(cuts, 40)
    bound = (cuts * 2.0 ** -22 + (adds + 1) * U) * size
    bound = bound + (want.abs() + bound) * (torch.finfo(out.dtype).eps / 2)
    off = (got - want).abs()
    assert (off <= bound).all(), float((off / bound.clamp(min=1e-300)).max())
    if out.dtype == FP32 and live:
        assert (got - want).norm() <= 1e-6 * want.norm()
    # other rows and the columns behind the results are left as they were
    assert out[live:].isnan().all() and out[:, n:].isnan().all()


SIZES = [([1], 8, 32), ([1, 0, 2], 16, 96), ([5, 1, 0, 9], 264, 512), ([3] * 8, 520, 2880),
         ([1] * 8, 4096, 4096), ([17, 40, 0, 3], 136, 1056), ([70, 1, 129], 1032, 288),
         ([256, 255, 257, 0, 1], 256, 544), ([193, 64, 32], 2056, 1024), ([600], 392, 768),
         ([0, 0], 64, 64), ([33] * 5, 128, 8192), ([300, 20], 120, 320), ([1000, 24], 48, 1248),
         ([12, 0, 1] + [0] * 13, 72, 352), ([1] * 40, 64, 128), ([513, 225], 264, 1120)]


@pytest.mark.parametrize("sizes,n,k", SIZES)
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_product(cuda_lib, sizes, n, k, fmt, dtype):
    for gather in (False, True):
        s = layer(sizes, n, k, fmt, gather=gather, extra=3, seed=n + k, factor=gather,
                  pad=int(gather))
        check(s, product(cuda_lib, s, dtype, ld=n + 8 * int(gather)))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 24, 63, 64, 65, 300])
def test_dense(cuda_lib, fmt, rows):
    """One matrix, no offsets; every row belongs to it."""
    s = layer([rows], 520, 1184, fmt, seed=rows)
    s["off"] = None
    for dtype in (BF16, FP32):
        check(s, product(cuda_lib, s, dtype))


@pytest.mark.parametrize("fmt", [MX, NV])
def test_many_tiles(cuda_lib, fmt):
    """More tiles for a pair of SMs than it lists at its start (64), gathered or not."""
    for gather, dtype in ((False, BF16), (True, BF16), (True, FP32)):
        s = layer([3, 1] * 32, 21 * 1024 + 8, 64, fmt, gather=gather, seed=4, extra=2, factor=True)
        check(s, product(cuda_lib, s, dtype))


@pytest.mark.parametrize("fmt", [MX, NV])
def test_long_sums(cuda_lib, fmt):
    """BF16 results of sums that leave the tensor cores on their way, and just not."""
    for k in (131072, 131104, 200032):
        for gather in (False, True):
            s = layer([40, 3], 72, k, fmt, gather=gather, seed=k)
            for dtype in (BF16, FP32):
                check(s, product(cuda_lib, s, dtype))


@pytest.mark.parametrize("fmt", [MX, NV])
def test_small_tiles_between_large_ones(cuda_lib, fmt):
    """Tiles that reach the columns both accumulators have, and tiles that do not, in any order;
    gathering warps without a row in between."""
    sizes = [256, 3, 200, 1, 256, 256, 40, 130, 5, 250, 0, 90, 255, 161, 209, 160, 208]
    for k in (64, 544, 2080):
        for gather in (False, True):
            s = layer(sizes * 3, 264, k, fmt, gather=gather, seed=k)
            check(s, product(cuda_lib, s, BF16))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows", [2, 40, 700])
def test_scales_far_apart(cuda_lib, fmt, rows):
    """Scales over the formats' ranges: sums of terms of very different size."""
    s = layer([rows, rows], 136, 512, fmt, seed=rows,
              scale_range=(80, 160) if fmt == MX else (0, 127))
    check(s, product(cuda_lib, s, FP32))


@pytest.mark.parametrize("rows", [3, 400])
@pytest.mark.parametrize("fmt,of_weight,of_x", [
    (MX, 0, 254), (MX, 254, 0), (MX, 0, 127), (MX, 1, 126), (MX, 64, 64), (MX, 250, 20),
    (MX, 127, 127), (NV, 0x01, 0x7E), (NV, 0x7E, 0x7E), (NV, 0x01, 0x01), (NV, 0, 0x38),
    (NV, 0xB8, 0x38), (NV, 0xB8, 0x81)])
def test_ends_of_the_scales(cuda_lib, rows, fmt, of_weight, of_x):
    """The smallest and largest scales, and E4M3 with the bit that is not used: sums of 256
    products of one pair of scales are exact."""
    s = layer([rows], 64, 256, fmt, seed=1)
    s["ws"].view(U8).fill_(of_weight)
    s["xs"].view(U8).fill_(of_x)
    out = product(cuda_lib, s, FP32)
    assert torch.equal(out.double(), exact(s)[0])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,gather", [(3, False), (400, False), (400, True)])
def test_the_bit_that_is_not_used(cuda_lib, rows, gather, dtype):
    """E4M3 scales of any code, NaN among them: with bit 7 set the results are the same."""
    s = layer([rows, rows], 72, 1184, NV, gather=gather, seed=rows, scale_range=(0, 127))
    s["xs"].view(U8)[1, 3] = 127
    s["ws"].view(U8)[1, 5, 2] = 127
    want = product(cuda_lib, s, dtype)
    assert want.isnan().any() and not want.isnan().all()
    for scales in (s["xs"], s["ws"]):
        scales.view(U8).bitwise_or_(torch.randint(0, 2, scales.shape, device="cuda", dtype=U8) * 128)
    s["xs"].view(U8)[1, 3] = 255
    s["ws"].view(U8)[1, 5, 2] = 255
    assert torch.equal(product(cuda_lib, s, dtype).nan_to_num(123.0), want.nan_to_num(123.0))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows", [3, 40, 400])
def test_one_nan_block(cuda_lib, fmt, rows):
    """A NaN scale reaches its row's results, or its column's, and no other."""
    s = layer([rows, rows], 72, 640, fmt, extra=2, seed=3)
    nan = 255 if fmt == MX else 127
    s["xs"].view(U8)[1, 3] = nan
    s["xs"].view(U8)[2 * rows:] = nan       # rows of no expert
    s["ws"].view(U8)[1, 5, 2] = nan
    out = product(cuda_lib, s, FP32)
    want = torch.zeros((2 * rows, 72), dtype=torch.bool, device="cuda")
    want[1] = True
    want[rows:, 5] = True
    assert torch.equal(out[:2 * rows].isnan(), want)
    fine = exact(s)[0][:2 * rows]
    got = out[:2 * rows].double()[~want]
    assert (got - fine[~want]).norm() <= 1e-6 * fine[~want].norm()


@pytest.mark.parametrize("rows", [6, 60, 900])
def test_offsets_that_do_not_fit(cuda_lib, rows):
    """Beyond the rows: cut; not ascending: no row is written."""
    s = layer([rows // 3] * 3, 64, 256, MX, seed=1)
    s["off"][3] = 2 ** 30
    s["sizes"][2] = rows - 2 * (rows // 3)
    check(s, product(cuda_lib, s, FP32))
    s["off"].copy_(torch.tensor([0, rows - 1, 1, rows]))
    assert product(cuda_lib, s, FP32).isnan().all()
    s["off"].copy_(torch.tensor([-5, -1, 0, 2]))
    s["sizes"] = [0, 0, 2]
    out = product(cuda_lib, s, FP32)
    check(s, out)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows", [7, 40])
def test_offsets_beyond_32_bits(cuda_lib, rows, fmt):
    """Rows so far apart that every operand's bytes pass 2^32 (the few rows' kernel and
    the other)."""
    E, n, k = 2, 72, 288

    def far(shape, width, dtype, total=2 ** 33):
        of = 1
        for d in shape:
            of *= d
        whole = torch.empty((*shape, total // of // 16 * 16), dtype=dtype, device="cuda")
        assert (of - 1) * whole.stride(-2) > 0.8 * total
        return whole[..., :width]

    s = layer([rows - 2, 2], n, k, fmt, seed=rows)
    x = far((rows,), k, BF16, 2 ** 32)
    x.copy_(torch.randn((rows, k), device="cuda"))
    codes, byte = fp4.quantize(x, fmt, None)
    for name, width in (("x", k // 2), ("xs", k // fp4.BLOCK[fmt])):
        s[name] = far((rows,), width, U8)
    s["xs"] = s["xs"].view(fmt)
    cuda_lib.moe_quantize_fp4(x, s["x"], s["xs"])
    assert torch.equal(s["x"], fp4.pack(codes)) and torch.equal(s["xs"].view(U8), byte)
    del x
    back = far((rows,), k, FP32, 2 ** 32)
    cuda_lib.moe_dequantize_fp4(s["x"], s["xs"], back)
    assert torch.equal(back.double(), fp4.values(s["x"], s["xs"]))
    del back
    for name in ("w", "ws"):
        t = far((E, n), s[name].shape[-1], U8)
        t.copy_(s[name].view(U8))
        s[name] = t.view(s[name].dtype)
    for dtype in (BF16, FP32):
        out = far((rows,), n + 8, dtype, 2 ** 32).fill_(NAN)
        cuda_lib.moe_grouped_gemm_fp4(s["x"], s["xs"], s["w"], s["ws"], s["off"], out[:, :n])
        check(s, out)
        del out
    s["index"] = torch.arange(rows - 1, -1, -1, device="cuda").int()
    out = far((rows,), n, FP32, 2 ** 32)
    cuda_lib.moe_grouped_gemm_fp4(s["x"], s["xs"], s["w"], s["ws"], s["off"], out,
                                  row_index=s["index"])
    check(s, out)
    del out, t, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", [MX, NV])
def test_results_do_not_depend_on_the_company(cuda_lib, fmt):
    """Passes repeat bit for bit, on other streams and in a replayed graph too."""
    for sizes in ([1] * 8, [90, 300, 7]):
        s = layer(sizes, 264, 1056, fmt, gather=True, seed=2, factor=True)
        first = product(cuda_lib, s, BF16)
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        outs = []
        for st in streams * 3:
            with torch.cuda.stream(st):
                outs.append(product(cuda_lib, s, BF16))
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o.nan_to_num(9.0), first.nan_to_num(9.0))
        out = torch.full_like(first, NAN)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cuda_lib.moe_grouped_gemm_fp4(s["x"], s["xs"], s["w"], s["ws"], s["off"], out,
                                          row_index=s["index"], factor=s["factor"])
        other = layer(sizes, 264, 1056, fmt, gather=True, seed=5, factor=True)
        for name in ("x", "w", "off", "index", "factor"):
            s[name].copy_(other[name])
        for name in ("xs", "ws"):
            s[name].view(U8).copy_(other[name].view(U8))
        graph.replay()
        torch.cuda.synchronize()
        check(s, out)


def test_layer_as_used(cuda_lib):
    """Permutation, quantisation, the gathered product, quantisation of its result, the second
    product and the weighted way back, against float64 of the same 4-bit values."""
    mf = cuda_lib
    T, K, E, H, N = 150, 4, 6, 544, 288
    g = torch.Generator().manual_seed(7)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int()
    ids[3] = -1
    ids = ids.cuda()
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    rw = torch.rand((T, K), generator=g).cuda()
    for fmt in (MX, NV):
        up = torch.randn((E * N, H), generator=g).bfloat16().cuda()
        down = torch.randn((E * H, N), generator=g).bfloat16().cuda()
        qx, qu, qd, qy = (mf.moe_fp4_empty(sh, k, fmt) for sh, k in
                          (((T,), H), ((E, N), H), ((E, H), N), ((T * K,), N)))
        mf.moe_quantize_fp4(x, *qx)
        mf.moe_quantize_fp4(up, qu[0].view(-1, H // 2), qu[1].flatten(0, 1))
        mf.moe_quantize_fp4(down, qd[0].view(-1, N // 2), qd[1].flatten(0, 1))
        off, idx, tok = mf.moe_expert_permutation(ids, E)
        n = int(off[E])
        y = torch.zeros((T * K, N), dtype=FP32, device="cuda")
        mf.moe_grouped_gemm_fp4(*qx, *qu, off, y, row_index=tok)
        mf.moe_quantize_fp4(y, *qy)
        z = torch.full((T * K, H), NAN, dtype=FP32, device="cuda")
        mf.moe_grouped_gemm_fp4(*qy, *qd, off, z)
        out = torch.empty((T, H), dtype=FP32, device="cuda")
        mf.moe_combine(z, rw, idx, out)
        expert = ids.flatten()[ids.flatten() >= 0].sort(stable=True).values.long()
        wu, wd = fp4.values(*qu), fp4.values(*qd)
        want = torch.einsum("rk,rnk->rn", fp4.values(*qx)[tok[:n].long()], wu[expert])
        assert (y[:n].double() - want).norm() <= 1e-6 * want.norm()
        want = torch.einsum("rk,rnk->rn", fp4.values(*qy)[:n], wd[expert])
        assert (z[:n].double() - want).norm() <= 1e-6 * want.norm()
        slot = idx.clamp(min=0).long()
        terms = torch.where((idx >= 0).unsqueeze(-1), want[slot], torch.zeros((), device="cuda",
                                                                               dtype=torch.float64))
        total = (terms * rw.double().unsqueeze(-1)).sum(1)
        assert (out.double() - total).norm() <= 2e-6 * total.norm()
