"""Timed cases of the expert-layer operators: the permutation by expert (and the
gradient of its gather), the matrix products grouped by expert (forward, both
gradients) and the products with 4-bit weights.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes a case's inputs on the GPU from a seed, ``run`` makes one
pass (the plain torch form, or with ``own`` the library's kernels) and
``exact`` gives the definition's result in float64.
"""
import math

import torch

own = False

BF16, FP32 = "bf16", "fp32"
_DTYPES = {BF16: torch.bfloat16, FP32: torch.float32}


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # the index map of a decode batch: 32 tokens, latency only
        dict(name="permute_decode", op="permute", tokens=32, top_k=8, experts=128, packed=False,
             dropped=0.0, skew=0.5),
        # the index map of a long prefill, from packed routing words, some slots on other ranks
        dict(name="permute_prefill", op="permute", tokens=32768, top_k=8, experts=256, packed=True,
             dropped=0.01, skew=0.5),
        # gradient of the gather: a short odd batch with FP32 rows
        dict(name="row_sum_odd", op="row_sum", tokens=517, top_k=6, experts=40, hidden=2056,
             dropped=0.05, skew=0.5, in_type=FP32, out_type=FP32),
        # gradient of the gather: a training batch at hidden 7168
        dict(name="row_sum_training", op="row_sum", tokens=8000, top_k=8, experts=64, hidden=7168,
             dropped=0.0, skew=0.5, in_type=BF16, out_type=BF16),
        # one decoded token through eight experts' first matrices: bound by the weights' bytes
        dict(name="gemm_one_token", op="gemm", tokens=1, top_k=8, experts=64, n=2048, k=4096,
             gather=True, dropped=0.0, skew=0.0, idle=0, out_type=BF16),
        # prefill of 4096 tokens through the gate-and-up matrices, rows gathered from the tokens
        dict(name="gemm_prefill", op="gemm", tokens=4096, top_k=8, experts=64, n=4096, k=4096,
             gather=True, dropped=0.0, skew=0.5, idle=0, out_type=BF16),
        # odd sizes, a strongly skewed router, idle experts, dropped slots, FP32 result
        dict(name="gemm_ragged", op="gemm", tokens=999, top_k=5, experts=30, n=1416, k=2200,
             gather=False, dropped=0.03, skew=1.2, idle=4, out_type=FP32),
        # training: the gradient of the rows
        dict(name="gemm_dgrad", op="dgrad", tokens=4096, top_k=8, experts=64, n=4096, k=2048,
             dropped=0.0, skew=0.5, idle=0, out_type=BF16),
        # training: the gradient of the weights, in FP32, rows gathered from the tokens
        dict(name="gemm_wgrad", op="wgrad", tokens=4096, top_k=8, experts=32, n=2048, k=4096,
             gather=True, dropped=0.0, skew=0.5, idle=1, out_type=FP32),
        # one decoded token through eight experts' 4-bit matrices
        dict(name="int4_one_token", op="int4", tokens=1, top_k=8, experts=64, n=4096, k=4096,
             group=128, zeros=False, gather=True, dropped=0.0, skew=0.0, idle=0,
             scale_type=BF16, out_type=BF16),
        # a decode batch of 64 tokens, small groups with zero points
        dict(name="int4_batch", op="int4", tokens=64, top_k=8, experts=64, n=4096, k=2048,
             group=32, zeros=True, gather=True, dropped=0.0, skew=0.3, idle=0,
             scale_type=BF16, out_type=BF16),
        # a dense 4-bit matrix with an odd number of rows, three vectors
        dict(name="int4_dense", op="int4", tokens=3, top_k=1, experts=1, n=20003, k=7168,
             group=64, zeros=False, gather=False, dropped=0.0, skew=0.0, idle=0,
             scale_type=FP32, out_type=FP32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["permute", "row_sum", "gemm", "gemm", "dgrad", "wgrad", "int4", "int4"])
    skew = rng.choice([0.0, 0.3, 0.5, 1.0, 1.3])
    dropped = rng.choice([0.0, 0.0, 0.02, 0.2])
    if op == "permute":
        experts = _log_int(rng, 2, 512)
        return dict(op=op, tokens=_log_int(rng, 1, 32768), top_k=rng.randint(1, min(8, experts)),
                    experts=experts, packed=rng.random() < 0.5, dropped=dropped, skew=skew)
    if op == "row_sum":
        experts = _log_int(rng, 8, 256)
        return dict(op=op, tokens=_log_int(rng, 1, 8000), top_k=rng.randint(1, 8), experts=experts,
                    hidden=8 * _log_int(rng, 32, 896), dropped=dropped, skew=skew,
                    in_type=rng.choice([BF16, FP32]), out_type=rng.choice([BF16, FP32]))
    experts = _log_int(rng, 4, 96)
    case = dict(op=op, tokens=0, top_k=rng.randint(1, min(8, experts)), experts=experts,
                n=0, k=0, gather=rng.random() < 0.5, dropped=dropped, skew=skew,
                idle=rng.choice([0, 0, experts // 8]), out_type=rng.choice([BF16, BF16, FP32]))
    case["top_k"] = min(case["top_k"], experts - case["idle"])
    if op == "int4":
        group = rng.choice([32, 64, 128])
        case.update(tokens=_log_int(rng, 1, 96), n=_log_int(rng, 500, 6000),
                    k=group * _log_int(rng, max(4, 512 // group), 7168 // group), group=group,
                    zeros=rng.random() < 0.5, scale_type=rng.choice([BF16, FP32]))
        return case
    case.update(n=8 * _log_int(rng, 32, 640), k=8 * _log_int(rng, 32, 640))
    if op == "dgrad":
        case["gather"] = False
    # from one token to as many as keep the product within a prefill's
    most = min(4096, int(5e11 / (2.0 * case["n"] * case["k"] * case["top_k"])))
    case["tokens"] = _log_int(rng, 1 if op == "gemm" else 64, max(most, 65))
    return case


# ---------------------------------------------------------------------------
# inputs

def _popularity(case):
    """How often the router picks each expert: a power law; the last `idle` experts never."""
    live = case["experts"] - case.get("idle", 0)
    w = [(1.0 + e) ** -case["skew"] for e in range(live)]
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


def _randn(shape, gen, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)
            if scale != 1.0 else torch.randn(shape, generator=gen, device="cuda", dtype=dtype))


def _activations(shape, gen):
    """N(0, 1) with one channel in 64 eight times as large, as hidden states have."""
    x = _randn(shape, gen)
    x[:, 5::64] *= 8
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "row_sum":
        s["map"] = _sort_by_expert(_route(case, gen), case["experts"])[1]
        rows = case["tokens"] * case["top_k"]
        s["permuted"] = _randn((rows, case["hidden"]), gen, dtype=_DTYPES[case["in_type"]])
        s["out"] = torch.zeros((case["tokens"], case["hidden"]), dtype=_DTYPES[case["out_type"]],
                               device="cuda")
        return s
    ids = _route(case, gen)
    if op == "permute":
        if case["packed"]:
            w = torch.rand(ids.shape, generator=gen, device="cuda").bfloat16()
            ids = (ids << 16) | (w.view(torch.int16).int() & 0xFFFF)
        s["ids"] = ids
        return s
    E, N, K = case["experts"], case["n"], case["k"]
    rows = ids.numel()
    offsets, _, tokens = _sort_by_expert(ids, E)
    s["offsets"] = offsets
    s["bounds"] = offsets.tolist()   # a plain program keeps the group sizes on the host
    gather = case.get("gather", False)
    s["index"] = tokens if gather else None
    out_type = _DTYPES[case["out_type"]]
    if op in ("gemm", "wgrad", "int4"):
        s["x"] = _activations((case["tokens"] if gather else rows, K), gen)
    if op in ("dgrad", "wgrad"):
        s["dy"] = _randn((rows, N), gen)
    if op in ("gemm", "dgrad"):
        s["w"] = _randn((E, N, K), gen, scale=K ** -0.5)
    if op == "int4":
        groups = K // case["group"]
        s["q"] = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda",
                               dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand((E, N, groups), generator=gen, device="cuda"))
                       * (K ** -0.5 / 4.6)).to(_DTYPES[case["scale_type"]])
        s["zeros"] = (torch.randint(5, 11, (E, N, groups), generator=gen, device="cuda",
                                    dtype=torch.uint8) if case["zeros"] else None)
        if case["experts"] == 1 and not gather and not case["dropped"]:
            s["offsets"] = None      # a dense matrix: every row
    shape = {"gemm": (rows, N), "int4": (rows, N), "dgrad": (rows, K), "wgrad": (E, N, K)}[op]
    s["out"] = torch.zeros(shape, dtype=out_type, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass

def _unpack(q):
    return torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float()


def _plain(s):
    op, case = s["op"], s["case"]
    if op == "permute":
        ids = s["ids"] >> 16 if case["packed"] else s["ids"]
        return _sort_by_expert(ids, case["experts"])
    out = s["out"]
    if op == "row_sum":
        m = s["map"].long()
        rows = s["permuted"][m.clamp(min=0)].float() * (m >= 0).unsqueeze(-1)
        out.copy_(rows.sum(1))
        return out
    for e in range(case["experts"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if op == "wgrad" and lo == hi:
            out[e] = 0
        if lo == hi:
            continue
        if op != "dgrad":
            x = (s["x"][lo:hi] if s["index"] is None else s["x"][s["index"][lo:hi].long()]).float()
        if op == "gemm":
            out[lo:hi] = x @ s["w"][e].float().t()
        elif op == "dgrad":
            out[lo:hi] = s["dy"][lo:hi].float() @ s["w"][e].float()
        elif op == "wgrad":
            out[e] = s["dy"][lo:hi].float().t() @ x
        else:
            q = _unpack(s["q"][e])
            z = 8.0 if s["zeros"] is None else s["zeros"][e].float().repeat_interleave(
                case["group"], dim=1)
            w = (q - z) * s["scales"][e].float().repeat_interleave(case["group"], dim=1)
            out[lo:hi] = x @ w.t()
    return out


def _own(s):
    import moe_finalize_rmsnorm_gb300 as mf
    op, case = s["op"], s["case"]
    if op == "permute":
        return mf.moe_expert_permutation(s["ids"], case["experts"], packed=case["packed"])
    if op == "row_sum":
        return mf.moe_permuted_row_sum(s["permuted"], s["map"], s["out"])
    if op == "gemm":
        return mf.moe_grouped_gemm(s["x"], s["w"], s["offsets"], s["out"], row_index=s["index"])
    if op == "dgrad":
        return mf.moe_grouped_gemm_dgrad(s["dy"], s["w"], s["offsets"], s["out"])
    if op == "wgrad":
        return mf.moe_grouped_gemm_wgrad(s["dy"], s["x"], s["offsets"], s["out"],
                                         row_index=s["index"])
    return mf.moe_grouped_gemv_int4(s["x"], s["q"], s["scales"], s["offsets"], s["out"],
                                    zeros=s["zeros"], row_index=s["index"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition, in float64

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "permute":
        ids = s["ids"].long()
        if case["packed"]:
            ids = ids.bitwise_right_shift(16)
        ids = ids.reshape(-1)
        # position = slots of lower experts + earlier slots of the same expert
        member = ids[:, None] == torch.arange(case["experts"], device="cuda")[None, :]
        before = member.int().cumsum(0, dtype=torch.int32)
        counts = before[-1].double()
        start = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
        inside = member.any(1)
        own_rank = (before * member).sum(1) - 1
        pos = torch.where(inside, start[ids.clamp(0, case["experts"] - 1)].long() + own_rank,
                          torch.full_like(ids, -1))
        tok = torch.full_like(ids, -1)
        slots = torch.arange(ids.numel(), device="cuda")
        tok[pos[inside]] = slots[inside].div(case["top_k"], rounding_mode="floor")
        return start.int(), pos.view(s["ids"].shape).int(), tok.int()
    if op == "row_sum":
        total = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["top_k"]):
            m = s["map"][:, j].long()
            total[m >= 0] += s["permuted"].index_select(0, m[m >= 0]).double()
        return total
    y = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
        r = torch.arange(a, b, device="cuda")
        src = r if s["index"] is None else s["index"].index_select(0, r).long()
        if op == "gemm":
            y[a:b] = torch.einsum("rk,nk->rn", s["x"].index_select(0, src).double(),
                                  s["w"][e].double())
        elif op == "dgrad":
            y[a:b] = torch.einsum("rn,nk->rk", s["dy"][a:b].double(), s["w"][e].double())
        elif op == "wgrad":
            y[e] = torch.einsum("rn,rk->nk", s["dy"][a:b].double(),
                                s["x"].index_select(0, src).double())
        elif a < b:
            N, K, G = case["n"], case["k"], case["group"]
            packed = s["q"][e].long()
            q = torch.empty((N, K), dtype=torch.float64, device="cuda")
            q[:, 0::2] = packed.remainder(16).double()
            q[:, 1::2] = packed.div(16, rounding_mode="floor").double()
            q = q.view(N, K // G, G)
            q = q - (8 if s["zeros"] is None else s["zeros"][e].double().unsqueeze(-1))
            w = (q * s["scales"][e].double().unsqueeze(-1)).view(N, K)
            y[a:b] = torch.einsum("rk,nk->rn", s["x"].index_select(0, src).double(), w)
    return y


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op, T, k = case["op"], case["tokens"], case["top_k"]
    slots = T * k * (1.0 - case["dropped"])
    if op == "permute":
        return {"bytes": 12 * T * k + 4 * (case["experts"] + 1), "flops": 0}
    size = {BF16: 2, FP32: 4}
    if op == "row_sum":
        H = case["hidden"]
        return {"bytes": slots * H * size[case["in_type"]] + T * H * size[case["out_type"]]
                + 4 * T * k, "flops": slots * H}
    E, N, K = case["experts"], case["n"], case["k"]
    # experts that get a row, on average
    live = sum(1.0 - (1.0 - min(1.0, k * p) * (1.0 - case["dropped"])) ** T
               for p in _popularity(case))
    out = size[case["out_type"]]
    x = (min(T, slots) if case.get("gather") else slots) * K * 2
    maps = 4 * (E + 1) + (4 * slots if case.get("gather") else 0)
    if op == "gemm":
        b = x + live * N * K * 2 + slots * N * out
    elif op == "dgrad":
        b = slots * N * 2 + live * N * K * 2 + slots * K * out
    elif op == "wgrad":
        b = x + slots * N * 2 + E * N * K * out
    else:
        per_group = size[case["scale_type"]] + (1 if case["zeros"] else 0)
        b = x + live * N * (K / 2 + K / case["group"] * per_group) + slots * N * out
    return {"bytes": b + maps, "flops": 2.0 * slots * N * K}
