"""The operators around 4-bit weights with group scales: what is timed, in a
plain form and by the library's kernels.

  linear   y = x W^T (+ bias), W[n, k] = s[n, k / g] (q[n, k] - z[n, k / g]):
           16-bit activations, 4-bit codes, a scale (and, with ``zeros``, a
           4-bit zero point) for each group of g along K.
  moe      a mixture-of-experts layer: router, top-k, softmax, the chosen
           experts' gated MLPs (weights as above) and their weighted sum.
  encode   the stored form (codes, scales, zero points) of a 16-bit weight.

``run`` computes them from elementary torch operations where ``own`` is
false, and calls the library where it is true.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _linear(name, M, N, K, group, dtype="bf16", zeros=False, bias=False):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "group": group, "dtype": dtype,
            "zeros": zeros, "bias": bias}


def _moe(name, M, K, F, E, topk, group, dtype="bf16", zeros=False, norm=True):
    return {"name": name, "op": "moe", "M": M, "K": K, "F": F, "E": E, "topk": topk, "group": group,
            "dtype": dtype, "zeros": zeros, "norm": norm}


def _encode(name, N, K, group, dtype="bf16", zeros=False):
    return {"name": name, "op": "encode", "N": N, "K": K, "group": group, "dtype": dtype, "zeros": zeros}


def listed():
    return [
        # one generated token through a square attention projection: latency
        _linear("linear_m1_square", 1, 2560, 2560, 128),
        # one token through a gate or up projection: the weight stream
        _linear("linear_m1_wide", 1, 9728, 2560, 128),
        # a few sequences decoded together, down projection of a converted
        # fp16 checkpoint with zero points and a bias
        _linear("linear_m5_deep_fp16", 5, 2560, 9728, 64, "fp16", True, True),
        # a ragged layer (rows and K no multiple of any tile), small groups
        _linear("linear_m13_ragged", 13, 1001, 2720, 32, "bf16", True),
        # a short prompt
        _linear("linear_m76_wide", 76, 9728, 2560, 128),
        # a long prompt, the same layer as the decoded one
        _linear("linear_m1220_deep", 1220, 2560, 9728, 128),
        # one token through an expert layer of many small experts: latency
        _moe("moe_m1_e128", 1, 2048, 768, 128, 8, 128),
        # a small decoding batch over the same layer
        _moe("moe_m16_e128", 16, 2048, 768, 128, 8, 128),
        # an odd batch, fp16 with zero points and small groups, raw softmax weights
        _moe("moe_m5_e60_fp16", 5, 1376, 1408, 60, 4, 32, "fp16", True, False),
        # few large experts, a full decoding batch: every expert is read
        _moe("moe_m64_e8", 64, 4096, 5632, 8, 2, 64),
        # a projection converted when a checkpoint is loaded
        _encode("encode_square", 2560, 2560, 128),
        # the gate weights of 32 experts in one call, zero points, small groups
        _encode("encode_experts", 32 * 1536, 2048, 32, "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "moe", "moe", "encode"])
    group = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    zeros = rng.random() < 0.5
    if op == "linear":
        while True:
            M, N = _log(rng, 1, 1220), _log(rng, 16, 12000)
            K = group * max(1, _log(rng, 256, 12000) // group)
            if M * N * K <= 1220 * 2560 * 9728:
                break
        return {"op": op, "M": M, "N": N, "K": K, "group": group, "dtype": dtype, "zeros": zeros,
                "bias": rng.random() < 0.5}
    if op == "moe":
        while True:
            E = rng.choice([8, 16, 60, 64, 128, 160])
            topk = rng.randint(1, 8)
            M = _log(rng, 1, 64)
            K = group * max(1, _log(rng, 512, 4096) // group)
            F = group * max(1, _log(rng, 256, 5632) // group)
            if E * K * F <= 8 * 4096 * 5632:
                break
        return {"op": op, "M": M, "K": K, "F": F, "E": E, "topk": topk, "group": group, "dtype": dtype,
                "zeros": zeros, "norm": rng.random() < 0.5}
    while True:
        N = _log(rng, 64, 50000)
        K = group * max(1, _log(rng, 256, 12000) // group)
        if N * K <= 32 * 1536 * 2048:
            break
    return {"op": op, "N": N, "K": K, "group": group, "dtype": dtype, "zeros": zeros}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _activations(gen, M, K, dtype):
    """N(0, 1) with half a percent of outlier channels, as after a norm."""
    x = torch.randn((M, K), generator=gen, device="cuda")
    n = max(1, round(0.005 * K))
    cols = torch.randperm(K, generator=gen, device="cuda")[:n]
    x[:, cols] *= 10.0
    return x.to(dtype)


def _stored(gen, shape, K, group, dtype, zeros):
    """Codes [*shape, K / 2] (two to a byte, even k in the low nibble), scales
    and zero points [*shape, K / group] of a weight of about N(0, 0.02)."""
    q = torch.randn((*shape, K), generator=gen, device="cuda", dtype=torch.float16).mul_(2.6).round_().add_(8)
    q = q.clamp_(0, 15).to(torch.uint8)
    codes = q[..., 0::2] | (q[..., 1::2] << 4)
    s = torch.randn((*shape, K // group), generator=gen, device="cuda").mul_(0.2).exp_().mul_(0.02 / 2.6).to(dtype)
    z = None
    if zeros:
        z = torch.randint(5, 12, (*shape, K // group), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, s, z


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)
    dtype, g, zeros = _DTYPES[case["dtype"]], case["group"], case["zeros"]
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        bias = None
        if case["bias"]:
            bias = torch.randn((N,), generator=gen, device="cuda").mul_(0.1).to(dtype)
        return {"x": _activations(gen, M, K, dtype), "w": _stored(gen, (N,), K, g, dtype, zeros), "bias": bias}
    if case["op"] == "moe":
        M, K, F, E = case["M"], case["K"], case["F"], case["E"]
        return {"x": _activations(gen, M, K, dtype),
                "router": torch.randn((E, K), generator=gen, device="cuda").mul_(1.5 / math.sqrt(K)).to(dtype),
                "gate": _stored(gen, (E, F), K, g, dtype, zeros),
                "up": _stored(gen, (E, F), K, g, dtype, zeros),
                "down": _stored(gen, (E, K), F, g, dtype, zeros)}
    w = torch.randn((case["N"], case["K"]), generator=gen, device="cuda").mul_(0.02)
    return {"weight": w.to(dtype)}


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import rotated_bit_quantized_convrot_amd as crp
        # laid out once, when the weights are loaded
        for name in ("w", "gate", "up", "down"):
            if name in state:
                state[name] = crp.pack_weight_w4g(*state[name])
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import rotated_bit_quantized_convrot_amd as crp
    c = state["case"]
    if c["op"] == "linear":
        return crp.linear_w4g(state["x"], state["w"], c["N"], c["group"], zeros=c["zeros"], bias=state["bias"])
    if c["op"] == "moe":
        y, ids, weights = crp.moe_w4g(state["x"], state["router"], state["gate"], state["up"], state["down"],
                                      c["F"], c["group"], c["topk"], zeros=c["zeros"], norm=c["norm"],
                                      routing=True)
        return {"y": y, "ids": ids, "weights": weights}
    codes, scales, zeros = crp.encode_w4g(state["weight"], c["group"], zeros=c["zeros"])
    return _values(codes & 15, codes >> 4, scales, zeros)


def _values(even, odd, scales, zeros):
    """The codes at even and odd k as the numbers they are, scales, zero points."""
    out = {"even": even, "odd": odd, "scales": scales}
    if zeros is not None:
        out["zeros"] = zeros
    return out


def _dequantise(stored, group):
    codes, s, z = stored
    q = torch.stack((codes & 15, codes >> 4), -1).view(*codes.shape[:-1], -1, group).float()
    q -= 8.0 if z is None else z.unsqueeze(-1).float()
    q *= s.unsqueeze(-1).float()
    return q.view(*codes.shape[:-1], -1)


def _run_plain(state):
    c = state["case"]
    if c["op"] == "linear":
        y = state["x"].float() @ _dequantise(state["w"], c["group"]).t()
        if state["bias"] is not None:
            y += state["bias"].float()
        return y.to(state["x"].dtype)
    if c["op"] == "moe":
        return _moe_plain(state, c)
    w = state["weight"].view(c["N"], -1, c["group"]).float()
    dtype = state["weight"].dtype
    # a divisor on the device: by a host scalar, a division turns into a product with its reciprocal
    levels = w.new_full((), 15.0 if c["zeros"] else 7.0)
    if c["zeros"]:
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        s = ((hi - lo) / levels).to(dtype)
        sf = s.float()
        z = torch.where(sf > 0, (-lo / sf).round().clamp(0, 15), 0.0)
        q = torch.where(sf.unsqueeze(-1) > 0, ((w / sf.unsqueeze(-1)).round() + z.unsqueeze(-1)).clamp(0, 15), 0.0)
        z = z.to(torch.uint8)
    else:
        s = (w.abs().amax(-1) / levels).to(dtype)
        sf = s.float()
        q = torch.where(sf.unsqueeze(-1) > 0, (w / sf.unsqueeze(-1)).round().clamp(-8, 7) + 8.0, 8.0)
        z = None
    q = q.to(torch.uint8).view(c["N"], c["K"])
    return _values(q[:, 0::2].contiguous(), q[:, 1::2].contiguous(), s, z)


def _moe_plain(state, c):
    x = state["x"]
    # 64-bit logits: which experts are chosen hangs on values next to a border
    logits = x.double() @ state["router"].double().t()
    ranked, order = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids = order[:, :c["topk"]]
    p = torch.exp((logits - ranked[:, :1]).float())
    chosen = torch.gather(p, 1, ids)
    weights = chosen / (chosen if c["norm"] else p).sum(-1, keepdim=True)
    M, K, g = x.shape[0], x.shape[1], c["group"]
    pick = (lambda s, i: tuple(None if t is None else t[i] for t in s))
    if M * c["topk"] <= 4 * c["E"]:
        # few pairs for so many experts: the weights of each pair's expert
        flat = ids.reshape(-1)
        xe = x.float().repeat_interleave(c["topk"], 0).unsqueeze(-1)
        a = torch.bmm(_dequantise(pick(state["gate"], flat), g), xe)
        b = torch.bmm(_dequantise(pick(state["up"], flat), g), xe)
        h = a / (1 + torch.exp(-a)) * b
        o = torch.bmm(_dequantise(pick(state["down"], flat), g), h).view(M, c["topk"], K)
        y = (o * weights.unsqueeze(-1)).sum(1)
    else:
        # every expert on every token, weighted by zero where it is not chosen
        dense = torch.zeros_like(p).scatter_(1, ids, weights)
        xt = x.float().t().contiguous()
        y = torch.zeros((K, M), device=x.device)
        for e in range(c["E"]):
            a = _dequantise(pick(state["gate"], e), g) @ xt
            b = _dequantise(pick(state["up"], e), g) @ xt
            h = a / (1 + torch.exp(-a)) * b * dense[:, e]
            y += _dequantise(pick(state["down"], e), g) @ h
        y = y.t().contiguous()
    return {"y": y.to(x.dtype), "ids": ids.to(torch.int32), "weights": weights}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def _weight_bytes(n, c):
    """n weights: 4-bit codes, a 16-bit scale a group, a 4-bit zero point."""
    return n / 2 + n / c["group"] * (2.5 if c["zeros"] else 2.0)


def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": _weight_bytes(N * K, c) + 2 * M * K + 2 * M * N + (2 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    if c["op"] == "moe":
        M, K, F, E, k = c["M"], c["K"], c["F"], c["E"], c["topk"]
        active = E * (1 - (1 - k / E) ** M)
        return {"bytes": _weight_bytes(active * 3 * F * K, c) + 2 * E * K + 4 * M * K + 8 * M * k,
                "flops": 2 * M * k * 3 * F * K + 2 * M * E * K}
    N, K = c["N"], c["K"]
    return {"bytes": 2 * N * K + N * K / 2 + N * K / c["group"] * (3 if c["zeros"] else 2), "flops": 4 * N * K}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _weight64(stored, g):
    codes, s, z = stored
    rows = codes.reshape(-1, codes.shape[-1]).to(torch.int32)
    w = torch.empty((rows.shape[0], 2 * rows.shape[1]), dtype=torch.float64, device=rows.device)
    w[:, 0::2] = (rows % 16).double()
    w[:, 1::2] = (rows // 16).double()
    zero = torch.full(s.shape, 8.0, device=s.device, dtype=torch.float64) if z is None else z.double()
    at = torch.arange(w.shape[1], device=w.device) // g
    w = (w - zero.reshape(rows.shape[0], -1)[:, at]) * s.double().reshape(rows.shape[0], -1)[:, at]
    return w.reshape(*codes.shape[:-1], -1)


def exact(case, seed):
    c, t = case, _inputs(case, seed)
    if c["op"] == "linear":
        y = torch.matmul(_weight64(t["w"], c["group"]), t["x"].double().t()).t().contiguous()
        return y if t["bias"] is None else y + t["bias"].double()
    if c["op"] == "moe":
        x = t["x"].double()
        logits = torch.matmul(t["router"].double(), x.t()).t().contiguous()
        # ties to the lower index: the sort by value keeps the order of equals
        ids = torch.argsort(-logits, dim=1, stable=True)[:, :c["topk"]]
        soft = torch.softmax(logits, 1).gather(1, ids)
        weights = soft / soft.sum(1, keepdim=True) if c["norm"] else soft
        y = torch.zeros_like(x)
        for e in sorted(set(ids.flatten().tolist())):
            m, r = torch.nonzero(ids == e, as_tuple=True)
            one = [tuple(None if v is None else v[e] for v in t[name]) for name in ("gate", "up", "down")]
            wg, wu, wd = (_weight64(s, c["group"]) for s in one)
            a = torch.matmul(wg, x[m].t().contiguous())
            h = a * torch.sigmoid(a) * torch.matmul(wu, x[m].t().contiguous())
            y.index_add_(0, m, torch.matmul(wd, h).t() * weights[m, r].unsqueeze(1))
        return {"y": y, "ids": None, "weights": weights}
    # the codes follow from the rounded scales, so only the scales have a value in 64 bits
    w = t["weight"].double().reshape(c["N"], -1, c["group"])
    if c["zeros"]:
        return {"even": None, "odd": None, "zeros": None,
                "scales": (torch.relu(w.max(-1).values) + torch.relu((-w).max(-1).values)) / 15}
    return {"even": None, "odd": None, "scales": w.abs().max(-1).values / 7}
