"""Timed cases of the rows' way into expert order and back (with the routing weights
and their gradients) and of the expert products in microscaled 4-bit floating point
(the quantisation and the product).

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes a case's inputs on the GPU from a seed, ``run`` makes one
pass (the plain torch form, or with ``own`` the library's kernels) and
``exact`` gives the definition's result in float64.

Formats: "mx" has blocks of 32 values with a power of two as their scale (E8M0),
"nv" blocks of 16 with a scale in E4M3; the values are E2M1, two to a byte.
"""
import math

import torch

own = False

BF16, FP32, PACKED = "bf16", "fp32", "packed"
MX, NV = "mx", "nv"
_DTYPES = {BF16: torch.bfloat16, FP32: torch.float32}
_BLOCK = {MX: 32, NV: 16}
_SCALE = {MX: torch.float8_e8m0fnu, NV: torch.float8_e4m3fn}
_MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # a decode batch's tokens into expert order: latency only
        dict(name="dispatch_decode", op="dispatch", tokens=24, top_k=8, experts=128, hidden=4096,
             dropped=0.0, weights=None, in_type=BF16, out_type=BF16),
        # a training batch into expert order, the routing weights applied on the way in
        dict(name="dispatch_training", op="dispatch", tokens=8000, top_k=8, experts=64,
             hidden=7168, dropped=0.0, weights=FP32, in_type=BF16, out_type=BF16),
        # back to the tokens: an odd batch in FP32, some slots on no expert
        dict(name="combine_odd", op="combine", tokens=517, top_k=6, experts=40, hidden=2056,
             dropped=0.05, weights=BF16, in_type=FP32, out_type=FP32),
        # back to the tokens: a long prefill, weights in the router's packed words
        dict(name="combine_prefill", op="combine", tokens=16384, top_k=8, experts=64, hidden=4096,
             dropped=0.0, weights=PACKED, in_type=BF16, out_type=BF16),
        # gradients of the way back: an odd FP32 batch
        dict(name="combine_grad_odd", op="combine_grad", tokens=1031, top_k=5, experts=24,
             hidden=2872, dropped=0.03, weights=FP32, in_type=FP32, out_type=FP32),
        # gradients of the way back: a training batch
        dict(name="combine_grad_training", op="combine_grad", tokens=8000, top_k=8, experts=64,
             hidden=7168, dropped=0.0, weights=BF16, in_type=BF16, out_type=BF16),
        # the rows of a decode batch to 4 bits (and to the values they stand for)
        dict(name="quantize_decode", op="quantize", rows=32, k=4096, format=MX, factor=False,
             in_type=BF16),
        # a prefill's rows to 4 bits with a scale of the whole tensor
        dict(name="quantize_prefill", op="quantize", rows=16384, k=7168, format=NV, factor=True,
             in_type=BF16),
        # one decoded token through eight experts' matrices: bound by the weights' bytes
        dict(name="fp4_one_token", op="fp4", tokens=1, top_k=8, experts=64, n=4096, k=4096,
             format=MX, gather=True, dropped=0.0, skew=0.0, idle=0, factor=False, out_type=BF16),
        # a decode batch of 64 tokens: a few rows for each expert
        dict(name="fp4_batch", op="fp4", tokens=64, top_k=8, experts=64, n=4096, k=2048,
             format=NV, gather=True, dropped=0.0, skew=0.3, idle=0, factor=True, out_type=BF16),
        # prefill of 4096 tokens through the gate-and-up matrices, rows gathered from the tokens
        dict(name="fp4_prefill", op="fp4", tokens=4096, top_k=8, experts=64, n=4096, k=4096,
             format=NV, gather=True, dropped=0.0, skew=0.5, idle=0, factor=True, out_type=BF16),
        # odd sizes, a strongly skewed router, idle experts, dropped slots, FP32 result
        dict(name="fp4_ragged", op="fp4", tokens=999, top_k=5, experts=30, n=1416, k=2208,
             format=MX, gather=False, dropped=0.03, skew=1.2, idle=4, factor=False,
             out_type=FP32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "quantize", "fp4", "fp4", "fp4"])
    if op == "quantize":
        k = 32 * _log_int(rng, 4, 224)
        return dict(op=op, rows=_log_int(rng, 1, 16384), k=k, format=rng.choice([MX, NV]),
                    factor=rng.random() < 0.5, in_type=rng.choice([BF16, BF16, FP32]))
    dropped = rng.choice([0.0, 0.0, 0.02, 0.2])
    if op != "fp4":
        weights = rng.choice([FP32, BF16, PACKED] + ([None] if op == "dispatch" else []))
        in_type = rng.choice([BF16, FP32])
        hidden = 8 * _log_int(rng, 32, 896)
        top_k = rng.randint(1, 8)
        most = min(8000, int(8000 * 8 * 7168 * 2 / (top_k * hidden * (4 if in_type == FP32 else 2))))
        return dict(op=op, tokens=_log_int(rng, 1, most), top_k=top_k,
                    experts=_log_int(rng, 8, 256), hidden=hidden, dropped=dropped, weights=weights,
                    in_type=in_type, out_type=rng.choice([BF16, FP32]))
    experts = rng.choice([1, _log_int(rng, 4, 96), _log_int(rng, 4, 96)])
    idle = rng.choice([0, 0, experts // 8])
    case = dict(op=op, tokens=0, top_k=rng.randint(1, min(8, experts - idle)), experts=experts,
                n=8 * _log_int(rng, 32, 640), k=32 * _log_int(rng, 8, 160),
                format=rng.choice([MX, NV]), gather=experts > 1 and rng.random() < 0.5,
                dropped=dropped if experts > 1 else 0.0, skew=rng.choice([0.0, 0.3, 0.5, 1.0, 1.3]),
                idle=idle, factor=rng.random() < 0.5, out_type=rng.choice([BF16, BF16, FP32]))
    # from one token to as many as keep the product within a prefill's
    most = min(4096, int(5e11 / (2.0 * case["n"] * case["k"] * case["top_k"])))
    case["tokens"] = _log_int(rng, 1, max(most, 65))
    return case


# ---------------------------------------------------------------------------
# inputs

def _popularity(case):
    """How often the router picks each expert: a power law; the last `idle` experts never."""
    live = case["experts"] - case.get("idle", 0)
    w = [(1.0 + e) ** -case.get("skew", 0.5) for e in range(live)]
    return [x / sum(w) for x in w]


def _route(case, gen):
    """Expert ids [tokens, top_k], distinct within a token (Gumbel top-k); dropped slots are -1."""
    p = torch.tensor(_popularity(case), device="cuda")
    T, K = case["tokens"], case["top_k"]
    u = torch.rand((T, p.numel()), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
    ids = (p.log() - (-u.log()).log()).topk(K, dim=1).indices.int()
    ids = ids[:, torch.randperm(K, generator=gen, device="cuda")]
    if case["dropped"]:
        ids[torch.rand((T, K), generator=gen, device="cuda") < case["dropped"]] = -1
    return ids.contiguous()


def _sort_by_expert(ids, experts):
    """(offsets [experts + 1], position of each slot or -1, token of each row or -1)."""
    flat = ids.flatten().long()
    live = (flat >= 0) & (flat < experts)
    key = torch.where(live, flat, torch.full_like(flat, experts))
    order = key.argsort(stable=True)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.bincount(key, minlength=experts + 1)[:experts].cumsum(0)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device=ids.device)
    pos = torch.where(live, rank, torch.full_like(rank, -1)).view(ids.shape)
    tokens = torch.where(live[order], order // ids.shape[1], torch.full_like(order, -1))
    return offsets.int(), pos.int(), tokens.int()


def _activations(shape, gen, dtype=torch.bfloat16):
    """N(0, 1) with one channel in 64 eight times as large, as hidden states have."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    x[:, 5::64] *= 8
    return x


def _fp4_buffers(shape, k, fmt):
    """Bytes [..., k / 2] and scales [..., k / block] whose rows begin at multiples of 16 bytes."""
    groups = k // _BLOCK[fmt]
    scales = torch.zeros((*shape, -(-groups // 16) * 16), dtype=torch.uint8, device="cuda")
    return (torch.zeros((*shape, k // 2), dtype=torch.uint8, device="cuda"),
            scales[..., :groups].view(_SCALE[fmt]))


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "quantize":
        s["x"] = _activations((case["rows"], case["k"]), gen, _DTYPES[case["in_type"]])
        # one factor that brings the tensor's largest values near the top of the formats
        s["factor"] = (448.0 * 6.0 / s["x"].float().abs().amax()).reshape(1) if case["factor"] else None
        s["quantized"], s["scales"] = _fp4_buffers((case["rows"],), case["k"], case["format"])
        s["values"] = torch.zeros((case["rows"], case["k"]), dtype=torch.bfloat16, device="cuda")
        return s
    ids = _route(case, gen)
    offsets, pos, tokens = _sort_by_expert(ids, case["experts"])
    T, K, rows = case["tokens"], case["top_k"], ids.numel()
    if op != "fp4":
        H, in_type, out_type = case["hidden"], _DTYPES[case["in_type"]], _DTYPES[case["out_type"]]
        s["map"] = pos
        if case["weights"] is not None:
            w = torch.randn((T, K), generator=gen, device="cuda").softmax(1)
            if case["weights"] == PACKED:
                w = (ids << 16) | (w.bfloat16().view(torch.int16).int() & 0xFFFF)
            s["weights"] = w.bfloat16() if case["weights"] == BF16 else w
        else:
            s["weights"] = None
        if op == "dispatch":
            s["x"] = _activations((T, H), gen, in_type)
            s["out"] = torch.zeros((rows, H), dtype=out_type, device="cuda")
            return s
        s["permuted"] = torch.randn((rows, H), generator=gen, device="cuda", dtype=in_type)
        if op == "combine":
            s["out"] = torch.zeros((T, H), dtype=out_type, device="cuda")
            return s
        s["dy"] = torch.randn((T, H), generator=gen, device="cuda", dtype=out_type)
        s["grad_permuted"] = torch.zeros((rows, H), dtype=in_type, device="cuda")
        s["grad_weights"] = torch.zeros((T, K), dtype=torch.float32, device="cuda")
        return s
    E, N, K, fmt = case["experts"], case["n"], case["k"], case["format"]
    s["offsets"] = None if E == 1 else offsets
    s["bounds"] = offsets.tolist()   # a plain program keeps the group sizes on the host
    s["index"] = tokens if case["gather"] else None
    x = _activations((T if case["gather"] else rows, K), gen)
    s["x"], s["x_scales"] = _fp4_buffers((x.shape[0],), K, fmt)
    codes, scales = _quantize(x, None, fmt)
    s["x"].copy_(_pack(codes))
    s["x_scales"].view(torch.uint8).copy_(scales.view(torch.uint8))
    s["w"], s["w_scales"] = _fp4_buffers((E, N), K, fmt)
    s["w"].copy_(torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda",
                               dtype=torch.uint8))
    # scales of weights near K ** -0.5 (mx), and of the size that a factor goes with (nv)
    lo, hi = (117, 121) if fmt == MX else (0x30, 0x50)
    s["w_scales"].view(torch.uint8).copy_(
        torch.randint(lo, hi, (E, N, K // _BLOCK[fmt]), generator=gen, device="cuda",
                      dtype=torch.uint8))
    s["factor"] = ((0.5 + torch.rand(E, generator=gen, device="cuda")) * K ** -0.5
                   if case["factor"] else None)
    s["out"] = torch.zeros((rows, N), dtype=_DTYPES[case["out_type"]], device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass

def _quantize(x, factor, fmt):
    """(codes in uint8, scales) of the rows of x."""
    v = x.float() if factor is None else x.float() * factor
    v = v.unflatten(-1, (-1, _BLOCK[fmt]))
    most = v.abs().amax(-1)
    if fmt == MX:
        # the largest power of two up to `most`, over the 4 that E2M1's largest binade begins at
        e = torch.where(most == 0, 0, (torch.frexp(most).exponent - 3 + 127).clamp(0, 254))
        scales = e.to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        scales = (most / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    # borders between neighbours are decided in 64 bits
    q = v.double() / scales.double().unsqueeze(-1)
    q = torch.where(scales.float().unsqueeze(-1) == 0, 0.0, q)
    m = q.abs()
    codes = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) +
             (m >= 3.5) + (m > 5.0))
    return (codes + 8 * torch.signbit(v)).to(torch.uint8).flatten(-2), scales


def _values(codes, scales, fmt):
    """What 4-bit codes and their scales stand for, in FP32."""
    table = torch.tensor(_MAGNITUDES + [-m for m in _MAGNITUDES], device=codes.device)
    return (table[codes.int()].unflatten(-1, (-1, _BLOCK[fmt])) *
            scales.float().unsqueeze(-1)).flatten(-2)


def _unpack(q):
    return torch.stack((q & 15, q >> 4), dim=-1).flatten(-2)


def _weights(s):
    """Routing weights in FP32."""
    if s["case"]["weights"] == PACKED:
        return (s["weights"] << 16).view(torch.float32)
    return s["weights"].float()


def _plain(s):
    op, case = s["op"], s["case"]
    if op == "quantize":
        codes, scales = _quantize(s["x"], s["factor"], case["format"])
        s["values"].copy_(_values(codes, scales, case["format"]))
        return s["values"], scales
    if op == "fp4":
        fmt, out = case["format"], s["out"]
        for e in range(case["experts"]):
            lo, hi = s["bounds"][e], s["bounds"][e + 1]
            if lo == hi:
                continue
            r = slice(lo, hi) if s["index"] is None else s["index"][lo:hi].long()
            x = _values(_unpack(s["x"][r]), s["x_scales"].view(torch.uint8)[r].view(_SCALE[fmt]), fmt)
            y = x @ _values(_unpack(s["w"][e]), s["w_scales"][e], fmt).t()
            out[lo:hi] = y if s["factor"] is None else y * s["factor"][e]
        return out
    m = s["map"].long()
    live = m >= 0
    if op == "dispatch":
        v = s["x"].float().unsqueeze(1).expand(*m.shape, -1)
        if s["weights"] is not None:
            v = v * _weights(s).unsqueeze(-1)
        s["out"][m[live]] = v[live].to(s["out"].dtype)
        return s["out"]
    rows = s["permuted"][m.clamp(min=0)].float() * live.unsqueeze(-1)
    w = _weights(s).unsqueeze(-1)
    if op == "combine":
        s["out"].copy_((rows * w).sum(1))
        return s["out"]
    dy = s["dy"].float().unsqueeze(1)
    s["grad_permuted"][m[live]] = (w * dy)[live].to(s["grad_permuted"].dtype)
    s["grad_weights"].copy_((rows * dy).sum(-1))
    return s["grad_permuted"], s["grad_weights"]


def _own(s):
    import moe_finalize_rmsnorm_gb300 as mf
    op = s["op"]
    if op == "quantize":
        mf.moe_quantize_fp4(s["x"], s["quantized"], s["scales"], factor=s["factor"])
        mf.moe_dequantize_fp4(s["quantized"], s["scales"], s["values"])
        return s["values"], s["scales"]
    if op == "fp4":
        return mf.moe_grouped_gemm_fp4(s["x"], s["x_scales"], s["w"], s["w_scales"], s["offsets"],
                                       s["out"], row_index=s["index"], factor=s["factor"])
    if op == "dispatch":
        return mf.moe_dispatch(s["x"], s["map"], s["out"], expert_weights=s["weights"])
    if op == "combine":
        return mf.moe_combine(s["permuted"], s["weights"], s["map"], s["out"])
    return mf.moe_combine_backward(s["dy"], s["permuted"], s["weights"], s["map"],
                                   s["grad_permuted"], s["grad_weights"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition, in float64

def _power_of_two(e):
    """2 ** e for whole e in float64, from the format's bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _binade(v):
    """The whole e of 2 ** e <= v < 2 ** (e + 1), for v > 0 in float64."""
    e = v.log2().round()
    return e - (_power_of_two(e) > v).double()


def _exact_quantize(x, factor, fmt):
    """(values, scales) in float64; the product with the factor is rounded to FP32, as defined."""
    v = x.double()
    if factor is not None:
        v = (v * factor.double()).float().double()
    v = v.reshape(v.shape[0], -1, _BLOCK[fmt])
    top = v.abs().max(dim=2, keepdim=True).values
    tiny = 2.0 ** -1000
    if fmt == MX:
        scale = _power_of_two((_binade(top.clamp(min=tiny)) - 2).clamp(-127, 127))
    else:
        want = top / 6
        quantum = _power_of_two(_binade(want.clamp(min=tiny)).clamp(min=-6) - 3)
        scale = ((want / quantum).round() * quantum).clamp(max=448)
    a = torch.where(scale > 0, v.abs() / scale, torch.zeros_like(v))
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    a = ((a / step).round() * step).clamp(max=6)
    return (a * v.sign() * scale).flatten(1), scale.squeeze(2)


def _exact_values(q, scales, fmt):
    q = q.long()
    code = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.int64, device=q.device)
    code[..., 0::2] = q.remainder(16)
    code[..., 1::2] = q.div(16, rounding_mode="floor")
    e, m = code.div(2, rounding_mode="floor").remainder(4), code.remainder(2).double()
    a = torch.where(e == 0, m / 2, (1 + m / 2) * _power_of_two(e - 1))
    a = torch.where(code >= 8, -a, a)
    return a * scales.double().repeat_interleave(_BLOCK[fmt], dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s["x"], s["factor"], case["format"])
    if op == "fp4":
        fmt = case["format"]
        y = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        x = _exact_values(s["x"], s["x_scales"], fmt)
        for e, (a, b) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
            if a == b:
                continue
            src = torch.arange(a, b, device="cuda")
            src = src if s["index"] is None else s["index"].index_select(0, src).long()
            w = _exact_values(s["w"][e], s["w_scales"][e], fmt)
            y[a:b] = torch.einsum("rk,nk->rn", x.index_select(0, src), w)
            if s["factor"] is not None:
                y[a:b] *= s["factor"][e].double()
        return y
    T, K = s["map"].shape
    w = s["weights"]
    if w is not None:
        w = (w.bitwise_and(0xFFFF) << 16).view(torch.float32) if case["weights"] == PACKED else w
        w = w.double()
    zeros = lambda name: torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if op == "dispatch":
        y = zeros("out")
    elif op == "combine":
        y = zeros("out")
    else:
        y, gw = zeros("grad_permuted"), zeros("grad_weights")
    for j in range(K):
        m = s["map"][:, j].long()
        t = torch.arange(T, device="cuda")[m >= 0]
        m = m[m >= 0]
        scale = 1.0 if w is None else w[t, j].unsqueeze(1)
        if op == "dispatch":
            y.index_copy_(0, m, s["x"].index_select(0, t).double() * scale)
        elif op == "combine":
            y.index_add_(0, t, s["permuted"].index_select(0, m).double() * scale)
        else:
            dy = s["dy"].index_select(0, t).double()
            y.index_copy_(0, m, dy * scale)
            gw[t, j] = torch.einsum("th,th->t", s["permuted"].index_select(0, m).double(), dy)
    return (y, gw) if op == "combine_grad" else y


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op = case["op"]
    size = {BF16: 2, FP32: 4, PACKED: 4, None: 0}
    if op == "quantize":
        n = case["rows"] * case["k"]
        packed = n / 2 + n / _BLOCK[case["format"]]
        # to 4 bits: rows in, codes and scales out; and back: both in, BF16 values out
        return {"bytes": n * size[case["in_type"]] + 2 * packed + 2 * n, "flops": 2.0 * n}
    T, k = case["tokens"], case["top_k"]
    slots = T * k * (1.0 - case["dropped"])
    if op != "fp4":
        H, i, o = case["hidden"], size[case["in_type"]], size[case["out_type"]]
        maps = T * k * (4 + size[case["weights"]])
        if op == "dispatch":
            return {"bytes": T * H * i + slots * H * o + maps, "flops": slots * H}
        if op == "combine":
            return {"bytes": slots * H * i + T * H * o + maps, "flops": 2 * slots * H}
        return {"bytes": T * H * o + 2 * slots * H * i + 4 * T * k + maps, "flops": 3 * slots * H}
    E, N, K = case["experts"], case["n"], case["k"]
    # experts that get a row, on average
    live = sum(1.0 - (1.0 - min(1.0, k * p) * (1.0 - case["dropped"])) ** T
               for p in _popularity(case))
    row = K / 2 + K / _BLOCK[case["format"]]
    b = ((min(T, slots) if case["gather"] else slots) * row + live * N * row +
         slots * N * size[case["out_type"]] + 4 * (E + 1) + (4 * slots if case["gather"] else 0))
    return {"bytes": b, "flops": 2.0 * slots * N * K}
