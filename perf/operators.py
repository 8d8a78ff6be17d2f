"""The operators around the adapter apply, as measurable cases: the root-mean-square norm that makes the
apply's x, the expert gate beside the learned router, the base product that makes the apply's y, and the
adapted projection that chains norm, product and apply.

``run`` computes a case in plain torch, or, with ``own`` true, through this package's calls.
"""

import math

import torch

own = False

LOWEST_AMAX = 2.0 ** -64  # rows whose largest value is below this are scaled as if it were this
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the norm before a decoder layer's projections, one sequence decoding (d = 4096 as in the
        # 4-modality and decode workloads): launch latency counts
        {"name": "norm_decode", "op": "norm", "N": 1, "d": 4096, "dtype": "bf16", "residual": True, "out": True, "fp8": False},
        # the same norm over a prefill of 8192 tokens (the top-k scaling workload) that feeds an
        # e4m3 base product and, in bf16, the adapters
        {"name": "norm_prefill_fp8", "op": "norm", "N": 8192, "d": 4096, "dtype": "bf16", "residual": True, "out": True, "fp8": True},
        # fp32, an odd width (rows that start off 16-byte boundaries), no residual: a router's input norm
        {"name": "norm_ragged_fp32", "op": "norm", "N": 1237, "d": 2049, "dtype": "fp32", "residual": False, "out": True, "fp8": False},
        # softmax gate over a hot set of 64 adapters, 32 sequences decoding, bf16 logits
        {"name": "gate_decode", "op": "gate", "N": 32, "K": 64, "k": 2, "dtype": "bf16", "score": "softmax", "bias": False, "groups": 1, "keep": 1, "group_top": 1, "renorm": True, "scale": 1.0},
        # sigmoid gate over 256 experts in 8 groups with a balance bias, a prefill's worth of tokens
        {"name": "gate_groups", "op": "gate", "N": 16384, "K": 256, "k": 8, "dtype": "fp32", "score": "sigmoid", "bias": True, "groups": 8, "keep": 4, "group_top": 2, "renorm": True, "scale": 2.5},
        # softmax with a bias over 60 experts (not a power of two), a ragged batch of bf16 logits
        {"name": "gate_ragged", "op": "gate", "N": 40961, "K": 60, "k": 6, "dtype": "bf16", "score": "softmax", "bias": True, "groups": 1, "keep": 1, "group_top": 1, "renorm": False, "scale": 1.0},
        # the base projection of one decoding token, y in fp32 for the apply: bound by reading W
        {"name": "linear_decode", "op": "linear", "N": 1, "d_in": 4096, "d_out": 4096, "dtype": "bf16", "y": "fp32", "bias": False, "act": "none", "residual": False},
        # a prefill through a square projection with everything in the epilogue
        {"name": "linear_prefill", "op": "linear", "N": 8192, "d_in": 4096, "d_out": 4096, "dtype": "bf16", "y": "bf16", "bias": True, "act": "silu", "residual": True},
        # an e4m3 MLP projection (2048 -> 6144, the learned-router workload's shape) with its activation
        {"name": "linear_mlp_fp8", "op": "linear", "N": 4096, "d_in": 2048, "d_out": 6144, "dtype": "e4m3", "y": "bf16", "bias": True, "act": "gelu_tanh", "residual": False},
        # fp32 with odd sizes everywhere: a small head on an odd width
        {"name": "linear_ragged_fp32", "op": "linear", "N": 257, "d_in": 1031, "d_out": 517, "dtype": "fp32", "y": "fp32", "bias": True, "act": "relu", "residual": True},
        # one adapted projection of 16 decoding sequences: e4m3 base weights, bf16 adapters of rank 16
        {"name": "step_decode_fp8", "op": "step", "N": 16, "d_in": 4096, "d_out": 4096, "dtype": "e4m3", "K": 8, "r": 16, "k": 1, "bias": False},
        # the same over a prefill at the learned-router workload's shape, two adapters a token
        {"name": "step_prefill", "op": "step", "N": 4096, "d_in": 2048, "d_out": 6144, "dtype": "bf16", "K": 4, "r": 16, "k": 2, "bias": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gate", "linear", "step"])
    if op == "norm":
        d = _log_int(rng, 64, 8192)
        d = d if rng.random() < 0.3 else max(64, d // 64 * 64)  # mostly model widths, some odd
        fp8 = rng.random() < 0.4
        return {"op": op, "N": min(_log_int(rng, 1, 16384), 8192 * 4096 // d), "d": d, "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "residual": rng.random() < 0.7, "out": not fp8 or rng.random() < 0.5, "fp8": fp8}
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 6, 8])
        per = rng.randint(max(4, 16 // groups), 256 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        return {"op": op, "N": _log_int(rng, 1, 16384), "K": groups * per, "k": rng.randint(1, min(8, keep * per)),
                "dtype": rng.choice(["bf16", "fp32"]), "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6,
                "groups": groups, "keep": keep, "group_top": rng.choice([1, 2]) if groups > 1 else 1,
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5])}
    if op == "linear":
        dtype = rng.choice(["bf16", "bf16", "e4m3", "fp32"])
        d_in, d_out = _log_int(rng, 128, 4096), _log_int(rng, 32, 4096)
        if rng.random() < 0.8:  # model widths; the rest are odd
            d_in, d_out = max(128, d_in // 64 * 64), max(32, d_out // 32 * 32)
        return {"op": op, "N": _log_int(rng, 1, 8192 if dtype != "fp32" else 1024), "d_in": d_in, "d_out": d_out, "dtype": dtype,
                "y": "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"]), "bias": rng.random() < 0.5,
                "act": rng.choice(["none", "relu", "silu", "gelu_tanh"]), "residual": rng.random() < 0.5}
    d_in, d_out = 64 * rng.randint(4, 64), 64 * rng.randint(4, 64)
    K = rng.choice([2, 4, 8, 16])
    return {"op": op, "N": _log_int(rng, 1, 4096), "d_in": d_in, "d_out": d_out, "dtype": rng.choice(["bf16", "e4m3"]),
            "K": K, "r": rng.choice([16, 32]), "k": rng.randint(1, 2), "bias": rng.random() < 0.5}


# ------------------------------------------------------------------------------------ inputs
def _type(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _quantised(v):
    """v [rows x columns] in e4m3 with one fp32 scale a row."""
    scale = v.abs().amax(dim=1).clamp_min(LOWEST_AMAX) / E4M3_MAX
    return (v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _activations(g, N, d):
    """Hidden states: unit normals with the few wide channels that decoder layers have."""
    x = _randn(g, N, d)
    return x * (1.0 + 15.0 * (torch.rand(d, generator=g, device="cuda") < 0.01))


def _empty(shape, dtype):
    return torch.empty(shape, device="cuda", dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op, N = case["op"], case["N"]
    if op == "norm":
        t, d = _type(case["dtype"]), case["d"]
        s["x"] = _activations(g, N, d).to(t)
        s["res"] = (2.0 * _randn(g, N, d)).to(t) if case["residual"] else None
        s["g"] = (1.0 + 0.1 * _randn(g, d)).to(t)
        s["eps"] = 1e-6
        s["bufs"] = {"sum_out": _empty((N, d), t) if case["residual"] else None, "out": _empty((N, d), t) if case["out"] else None,
                     "out8": _empty((N, d), torch.float8_e4m3fn) if case["fp8"] else None,
                     "scale8": _empty((N,), torch.float32) if case["fp8"] else None}
    elif op == "gate":
        K = case["K"]
        s["logits"] = (1.5 * _randn(g, N, K) + 0.5 * _randn(g, K)).to(_type(case["dtype"]))
        s["b"] = 0.05 * _randn(g, K) if case["bias"] else None
        s["bufs"] = {"ids": _empty((N, case["k"]), torch.int32), "w": _empty((N, case["k"]), torch.float32)}
    else:
        d_in, d_out = case["d_in"], case["d_out"]
        W = _randn(g, d_out, d_in) / math.sqrt(d_in)
        s["b"] = 0.5 * _randn(g, d_out) if case["bias"] else None
        s["W"], s["sw"] = _quantised(W) if case["dtype"] == "e4m3" else (W.to(_type(case["dtype"])), None)
        if op == "linear":
            x = _randn(g, N, d_in)
            s["x"], s["sx"] = _quantised(x) if case["dtype"] == "e4m3" else (x.to(_type(case["dtype"])), None)
            t = _type(case["y"])
            s["res"] = _randn(g, N, d_out).to(t) if case["residual"] else None
            s["y"] = _empty((N, d_out), t)
        else:
            K, r, k = case["K"], case["r"], case["k"]
            s["x"], s["res"] = _activations(g, N, d_in).bfloat16(), (2.0 * _randn(g, N, d_in)).bfloat16()
            s["g"], s["eps"], s["scale"] = (1.0 + 0.1 * _randn(g, d_in)).bfloat16(), 1e-6, 2.0
            s["A"], s["B"] = (_randn(g, K, d_in, r) / math.sqrt(d_in)).bfloat16(), (_randn(g, K, r, d_out) / math.sqrt(r)).bfloat16()
            s["ids"] = torch.rand(N, K, generator=g, device="cuda").argsort(dim=1)[:, :k].to(torch.int32).contiguous()
            s["w"] = torch.softmax(_randn(g, N, k), dim=1)
            order = torch.argsort(s["ids"].reshape(-1), stable=True).to(torch.int32)  # the dispatch of ids, which the layer's projections share
            counts = torch.bincount(s["ids"].reshape(-1).long(), minlength=K)
            offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
            s["dispatch"] = (counts.to(torch.int32), offsets.to(torch.int32), order)
            fp8 = case["dtype"] == "e4m3"
            s["y"] = _empty((N, d_out), torch.bfloat16)
            s["bufs"] = {"sum_out": _empty((N, d_in), torch.bfloat16), "h": _empty((N, d_in), torch.bfloat16),
                         "h8": _empty((N, d_in), torch.float8_e4m3fn) if fp8 else None,
                         "scale8": _empty((N,), torch.float32) if fp8 else None}
    return s


# ------------------------------------------------------------------------------------ the passes
def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "gate": _plain_gate, "linear": _plain_linear, "step": _plain_step}[state["op"]](state)


def _own(s):
    import token_adapter_routing_gb300 as m
    if s["op"] == "norm":
        b = s["bufs"]
        m.molora_rmsnorm(s["x"], s["g"], s["eps"], residual=s["res"], **b)
        return [v for v in (b["sum_out"], b["out"], b["out8"], b["scale8"]) if v is not None]
    if s["op"] == "gate":
        return m.molora_gate_topk(s["logits"], s["k"], score=s["score"], bias=s["b"], groups=s["groups"], keep_groups=s["keep"],
                                  group_top=s["group_top"], renormalise=s["renorm"], scale=s["scale"], **s["bufs"])
    if s["op"] == "linear":
        return m.molora_linear(s["x"], s["W"], y=s["y"], x_scale=s["sx"], w_scale=s["sw"], bias=s["b"], act=s["act"], residual=s["res"])
    counts, offsets, perm = s["dispatch"]
    b = s["bufs"]
    m.molora_norm_linear_lora_apply(s["x"], s["g"], s["eps"], s["W"], s["A"], s["B"], s["ids"], s["y"], s["scale"], w=s["w"],
                                    counts=counts, offsets=offsets, perm=perm, residual=s["res"], w_scale=s["sw"], bias=s["b"], **b)
    return [s["y"], b["sum_out"], b["h"]]


def _norm(x, res, g, eps):
    v = x.float() if res is None else x.float() + res.float()
    return v, v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps) * g.float()


def _to_fp8(n):
    scale = n.abs().amax(dim=1).clamp_min(LOWEST_AMAX) / E4M3_MAX
    return (n / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    v, n = _norm(s["x"], s["res"], s["g"], s["eps"])
    out = [v.to(s["x"].dtype)] if s["residual"] else []
    if s["out"]:
        out.append(n.to(s["x"].dtype))
    if s["fp8"]:
        out += _to_fp8(n)
    return out


def _plain_gate(s):
    # scores in 32 bits, with the softmax's sum in 64 rounded once: its last bit decides between
    # experts whose biased scores nearly tie
    l, K, G = s["logits"].float(), s["K"], s["groups"]
    if s["score"] == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        score = e / e.double().sum(dim=1, keepdim=True).float()
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    by_logit = s["b"] is None and (G == 1 or s["group_top"] == 1)
    c = l if by_logit else score + s["b"] if s["b"] is not None else score
    if G > 1:
        best = c.view(-1, G, K // G).sort(dim=2, descending=True).values[:, :, :s["group_top"]]
        group = best[:, :, 0] if s["group_top"] == 1 else best[:, :, 0] + best[:, :, 1]
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, group.sort(dim=1, descending=True, stable=True).indices[:, :s["keep"]], True)
        c = c.masked_fill(~kept.repeat_interleave(K // G, dim=1), float("-inf"))
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    w = score.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), w * s["scale"]


def _act(v, name):
    if name == "relu":
        return v.clamp_min(0.0)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)
        return v / (1.0 + torch.exp(-2.0 * u))
    return v


def _product(x, W, sx, sw):
    v = x.float() @ W.float().t()
    return v if sx is None else v * sx[:, None] * sw[None, :]


def _plain_linear(s):
    v = _product(s["x"], s["W"], s["sx"], s["sw"])
    v = _act(v if s["b"] is None else v + s["b"], s["act"])
    return (v if s["res"] is None else v + s["res"].float()).to(_type(s["y"]) if isinstance(s["y"], str) else s["y"].dtype)


def _adapters(h, A, B, ids, w, scale):
    """scale * sum_j w[t,j] (h A_ids[t,j]) B_ids[t,j], over all adapters with weight 0 for the others."""
    K, r, d_out = B.shape
    c = torch.zeros(h.shape[0], K, device=h.device, dtype=h.dtype).scatter_add_(1, ids.long(), w.to(h.dtype))
    low = (h @ A.to(h.dtype).permute(1, 0, 2).reshape(h.shape[1], K * r)).view(-1, K, r) * c[:, :, None]
    return scale * (low.reshape(-1, K * r) @ B.to(h.dtype).reshape(K * r, d_out))


def _plain_step(s):
    v, n = _norm(s["x"], s["res"], s["g"], s["eps"])
    h = n.bfloat16()
    if s["sw"] is None:
        y = _product(h, s["W"], None, None)
    else:
        y = _product(*_swap(_to_fp8(n), s["W"]), s["sw"])
    y = y if s["b"] is None else y + s["b"]
    return [(y + _adapters(h.float(), s["A"], s["B"], s["ids"], s["w"], s["scale"])).bfloat16(), v.bfloat16(), h]


def _swap(quantised, W):
    return quantised[0], W, quantised[1]


# ------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"bf16": 2, "fp32": 4, "e4m3": 1}
    N = case["N"]
    if case["op"] == "norm":
        n = N * case["d"]
        b = size[case["dtype"]]
        each = b * (1 + 2 * case["residual"] + case["out"]) + case["fp8"]
        return {"bytes": n * each + b * case["d"] + 4 * N * case["fp8"], "flops": 6 * n}
    if case["op"] == "gate":
        return {"bytes": N * case["K"] * size[case["dtype"]] + 4 * case["K"] * case["bias"] + 8 * N * case["k"], "flops": 4 * N * case["K"]}
    d_in, d_out, b = case["d_in"], case["d_out"], size[case["dtype"]]
    scales = 4 * (N + d_out) if case["dtype"] == "e4m3" else 0
    if case["op"] == "linear":
        return {"bytes": b * d_in * (N + d_out) + scales + 4 * d_out * case["bias"] + size[case["y"]] * N * d_out * (1 + case["residual"]),
                "flops": 2 * N * d_in * d_out}
    K, r, k = case["K"], case["r"], case["k"]
    used = min(K, N * k)  # no more adapters are read than tokens choose
    return {"bytes": 2 * 4 * N * d_in + b * d_in * d_out + scales + 2 * used * r * (d_in + d_out) + 4 * d_out * case["bias"] + 2 * N * d_out + 8 * N * k,
            "flops": 2 * N * d_in * d_out + 2 * N * k * r * (d_in + d_out)}


# ------------------------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "gate":
        return _exact_gate(s)
    if case["op"] == "linear":
        acc = torch.matmul(s["x"].to(f), s["W"].to(f).T)
        if s["sx"] is not None:
            acc = acc * torch.outer(s["sx"].to(f), s["sw"].to(f))
        if s["b"] is not None:
            acc = acc + s["b"].to(f)
        if case["act"] == "relu":
            acc = torch.relu(acc)
        elif case["act"] == "silu":
            acc = acc * torch.sigmoid(acc)
        elif case["act"] == "gelu_tanh":
            acc = 0.5 * acc * (1 + torch.tanh(math.sqrt(2 / math.pi) * (acc + 0.044715 * acc ** 3)))
        return acc if s["res"] is None else acc + s["res"].to(f)
    total = s["x"].to(f)
    if s["res"] is not None:
        total = total + s["res"].to(f)
    normed = total / torch.sqrt(total.pow(2).mean(1, keepdim=True) + s["eps"]) * s["g"].to(f)
    if case["op"] == "norm":
        out = [total] if case["residual"] else []
        if case["out"]:
            out.append(normed)
        if case["fp8"]:
            scale8 = torch.clamp(normed.abs().max(1).values, min=LOWEST_AMAX) / E4M3_MAX
            out += [normed / scale8[:, None], scale8]
        return out
    h = normed.bfloat16().to(f)  # the products read the norm's row as it is stored
    if s["sw"] is None:
        base = torch.matmul(h, s["W"].to(f).T)
    else:
        scale8 = torch.clamp(normed.abs().max(1, keepdim=True).values, min=LOWEST_AMAX) / E4M3_MAX
        h8 = torch.clamp(normed / scale8, -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).to(f)
        base = torch.matmul(h8 * scale8, (s["W"].to(f) * s["sw"].to(f)[:, None]).T)
    if s["b"] is not None:
        base = base + s["b"].to(f)
    for a in range(case["K"]):
        weight = (s["w"].to(f) * (s["ids"] == a)).sum(1, keepdim=True)
        base = base + s["scale"] * weight * torch.matmul(torch.matmul(h, s["A"][a].to(f)), s["B"][a].to(f))
    return [base, total, normed]


def _exact_gate(s):
    """The weights of the experts that the definition selects (scores rounded to 32 bits are what it
    compares, ties go to the lower index); which ones is a matter of whole numbers."""
    N, K, G, k = s["N"], s["K"], s["groups"], s["k"]
    l = s["logits"].double()
    score = torch.softmax(l, 1) if s["score"] == "softmax" else torch.sigmoid(l)
    c = score.float() if s["b"] is None else score.float() + s["b"]
    if G > 1:
        rank = torch.topk(c.reshape(N, G, K // G), s["group_top"], dim=2).values.sum(2)
        place = torch.argsort(torch.argsort(-rank, dim=1, stable=True), dim=1)
        c = torch.where((place < s["keep"]).repeat_interleave(K // G, dim=1), c, torch.full_like(c, -math.inf))
    w = score.gather(1, torch.argsort(-c, dim=1, stable=True)[:, :k])
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return [None, w * s["scale"]]
