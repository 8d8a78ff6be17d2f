"""The feed-forward half of a layer, as measurable cases: the product in e4m3 with a scale for each block of 128,
the quantiser that makes its x, and the gated feed-forward block, both for serving (single tokens to prefills, bf16
and e4m3) and for training (forward and backward).

``run`` computes a case in plain torch, or, with ``own`` true, through this package's calls.
"""

import math

import torch

own = False

BLOCK = 128               # columns (and, of weights, rows) that share a scale
LOWEST_AMAX = 2.0 ** -64  # blocks whose largest value is below this are scaled as if it were this
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the activations of 16 sequences decoding (d = 4096 as in the 4-modality and decode workloads), on their
        # way into an e4m3 product: launch latency counts
        {"name": "quantise_decode", "op": "quantise", "N": 16, "d": 4096, "dtype": "bf16"},
        # the same for a prefill of 8192 tokens (the top-k scaling workload's batch)
        {"name": "quantise_prefill", "op": "quantise", "N": 8192, "d": 4096, "dtype": "bf16"},
        # fp32 activations of a ragged batch whose width ends inside a block
        {"name": "quantise_ragged_fp32", "op": "quantise", "N": 1237, "d": 2064, "dtype": "fp32"},
        # the block-scaled projection of one decoding token, y in fp32 for the adapters' apply: bound by reading W
        {"name": "blocks_decode", "op": "blocks", "N": 1, "d_in": 4096, "d_out": 4096, "y": "fp32", "bias": False, "act": "none", "residual": False},
        # a prefill through a square projection, the residual added in the epilogue (a feed-forward's way down)
        {"name": "blocks_prefill", "op": "blocks", "N": 8192, "d_in": 4096, "d_out": 4096, "y": "bf16", "bias": False, "act": "none", "residual": True},
        # sizes that end inside blocks and tiles, rows of y that start anywhere, everything in the epilogue
        {"name": "blocks_ragged", "op": "blocks", "N": 1237, "d_in": 2064, "d_out": 1541, "y": "fp32", "bias": True, "act": "silu", "residual": True},
        # the feed-forward block of one decoding token (2048 -> 6144, the learned-router workload's shape): bound by
        # reading both projections' weights
        {"name": "gated_decode", "op": "gated", "N": 1, "d_in": 2048, "d_ff": 6144, "dtype": "bf16", "act": "silu"},
        # the same over that workload's batch
        {"name": "gated_prefill", "op": "gated", "N": 4096, "d_in": 2048, "d_ff": 6144, "dtype": "bf16", "act": "silu"},
        # 32 sequences decoding through block-scaled e4m3 weights
        {"name": "gated_decode_fp8", "op": "gated", "N": 32, "d_in": 2048, "d_ff": 6144, "dtype": "e4m3", "act": "silu"},
        # the workload's batch through block-scaled e4m3 weights, the tanh form of GELU as the gate
        {"name": "gated_prefill_fp8", "op": "gated", "N": 4096, "d_in": 2048, "d_ff": 6144, "dtype": "e4m3", "act": "gelu_tanh"},
        # a training step of the block over that batch: forward, and the gradients of x and of the weights
        {"name": "train_step", "op": "train", "N": 4096, "d_in": 2048, "d_ff": 6144, "act": "silu"},
        # a small block over a ragged batch, with a width that no tile divides and that is odd
        {"name": "train_ragged", "op": "train", "N": 777, "d_in": 1032, "d_ff": 1365, "act": "gelu_tanh"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step, often=64):
    """A width between lo and hi: mostly a model's (a multiple of `often`), else any multiple of `step`."""
    step = often if rng.random() < 0.6 else step
    return max(lo, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["quantise", "blocks", "gated", "gated", "train"])
    if op == "quantise":
        d = _width(rng, 64, 8192, 1)
        return {"op": op, "N": min(_log_int(rng, 1, 16384), 8192 * 4096 // d), "d": d, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "blocks":
        return {"op": op, "N": _log_int(rng, 1, 8192), "d_in": _width(rng, 128, 4096, 16), "d_out": _width(rng, 32, 4096, 1),
                "y": rng.choice(["bf16", "fp32"]), "bias": rng.random() < 0.5, "act": rng.choice(["none", "relu", "silu", "gelu_tanh"]),
                "residual": rng.random() < 0.5}
    act = rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"])
    dtype = rng.choice(["bf16", "e4m3"]) if op == "gated" else "bf16"
    d_in, d_ff = _width(rng, 128, 4096, 16 if dtype == "e4m3" else 8), _width(rng, 64, 6144, 1)
    N = min(_log_int(rng, 1 if op == "gated" else 16, 8192), 4096 * 2048 * 6144 // (d_in * d_ff))
    case = {"op": op, "N": N, "d_in": d_in, "d_ff": d_ff, "act": act}
    return {**case, "dtype": dtype} if op == "gated" else case


# ------------------------------------------------------------------------------------ inputs
def _type(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, N, d):
    """Hidden states: unit normals with the few wide channels that decoder layers have."""
    x = _randn(g, N, d)
    return x * (1.0 + 15.0 * (torch.rand(d, generator=g, device="cuda") < 0.01))


def _spread(scale, rows, cols):
    """One value for each block, for each element: scale [rows or blocks of rows x blocks of columns]."""
    if scale.shape[0] != rows:
        scale = scale.repeat_interleave(BLOCK, dim=0)[:rows]
    return scale.repeat_interleave(BLOCK, dim=1)[:, :cols]


def _quantised_rows(v):
    """v [N x d] in e4m3, one scale for each row's block of 128 columns."""
    N, d = v.shape
    amax = torch.nn.functional.pad(v.abs(), (0, _blocks(d) * BLOCK - d)).view(N, _blocks(d), BLOCK).amax(dim=2)
    scale = amax.clamp_min(LOWEST_AMAX) / E4M3_MAX
    return (v / _spread(scale, N, d)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _quantised_weights(W):
    """W [d_out x d_in] in e4m3, one scale for each block of 128 x 128."""
    R, C = W.shape
    r, c = _blocks(R), _blocks(C)
    amax = torch.nn.functional.pad(W.abs(), (0, c * BLOCK - C, 0, r * BLOCK - R)).view(r, BLOCK, c, BLOCK).amax(dim=3).amax(dim=1)
    scale = amax.clamp_min(LOWEST_AMAX) / E4M3_MAX
    each = scale.repeat_interleave(BLOCK, dim=0)[:R].repeat_interleave(BLOCK, dim=1)[:, :C]
    return (W / each).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _empty(shape, dtype):
    return torch.empty(shape, device="cuda", dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op, N = case["op"], case["N"]
    if op == "quantise":
        d = case["d"]
        s["x"] = _activations(g, N, d).to(_type(case["dtype"]))
        s["bufs"] = {"out8": _empty((N, d), torch.float8_e4m3fn), "scale8": _empty((N, _blocks(d)), torch.float32)}
    elif op == "blocks":
        d_in, d_out = case["d_in"], case["d_out"]
        s["x"], s["sx"] = _quantised_rows(_activations(g, N, d_in))
        s["W"], s["sw"] = _quantised_weights(_randn(g, d_out, d_in) / math.sqrt(d_in))
        s["b"] = 0.5 * _randn(g, d_out) if case["bias"] else None
        t = _type(case["y"])
        s["res"] = (2.0 * _randn(g, N, d_out)).to(t) if case["residual"] else None
        s["buf"] = _empty((N, d_out), t)
    else:
        d_in, d_ff = case["d_in"], case["d_ff"]
        x = _randn(g, N, d_in)  # (a norm's output)
        Wg, Wu = _randn(g, d_ff, d_in) / math.sqrt(d_in), _randn(g, d_ff, d_in) / math.sqrt(d_in)
        s["sx"] = s["sw"] = None
        if case.get("dtype") == "e4m3":
            s["x"], s["sx"] = _quantised_rows(x)
            (g8, gs), (u8, us) = _quantised_weights(Wg), _quantised_weights(Wu)
            s["W"], s["sw"] = torch.cat([g8, u8]), torch.cat([gs, us])
        else:
            s["x"], s["W"] = x.bfloat16(), torch.cat([Wg, Wu]).bfloat16()
        s["h"] = _empty((N, d_ff), torch.bfloat16)
        if op == "train":
            s["dh"] = (_randn(g, N, d_ff) / math.sqrt(N)).bfloat16()
            s["proj"] = _empty((N, 2, (d_ff + 7) // 8 * 8), torch.bfloat16)
            s["dx"], s["dW"] = torch.empty_like(s["x"]), torch.empty_like(s["W"])
    return s


# ------------------------------------------------------------------------------------ the passes
def run(state):
    if own:
        return _own(state)
    return {"quantise": _plain_quantise, "blocks": _plain_blocks, "gated": _plain_gated, "train": _plain_train}[state["op"]](state)


def _own(s):
    import token_adapter_routing_gb300 as m
    if s["op"] == "quantise":
        return m.molora_quantise_blocks(s["x"], **s["bufs"])
    if s["op"] == "blocks":
        return m.molora_linear_blocks(s["x"], s["sx"], s["W"], s["sw"], y=s["buf"], bias=s["b"], act=s["act"], residual=s["res"])
    if s["op"] == "gated":
        return m.molora_gated_linear(s["x"], s["W"], h=s["h"], act=s["act"], x_scale=s["sx"], w_scale=s["sw"])
    h = m.molora_gated_linear(s["x"], s["W"], h=s["h"], act=s["act"])
    dx, dW, _ = m.molora_gated_linear_backward(s["x"], s["W"], s["dh"], act=s["act"], dx=s["dx"], dW=s["dW"], dproj=s["proj"])
    return [h, dx, dW]


def _plain_quantise(s):
    return _quantised_rows(s["x"].float())


def _act(v, name):
    if name == "relu":
        return v.clamp_min(0.0)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _slope(v, name):
    """The activation's derivative."""
    if name == "relu":
        return (v > 0.0).to(v.dtype)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    if name == "gelu":
        return 0.5 * torch.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        p = 1.0 / (1.0 + torch.exp(-c * (v + 0.044715 * v * v * v)))
        return p + v * p * (1.0 - p) * c * (1.0 + 3.0 * 0.044715 * v * v)
    return torch.ones_like(v)


def _weights(s):
    """The operands in 32 bits, gate and up rows apart."""
    F = s["d_ff"]
    if s["sx"] is None:
        return s["x"].float(), s["W"][:F].float(), s["W"][F:].float()
    N, d = s["x"].shape
    half = _blocks(F)
    return (s["x"].float() * _spread(s["sx"], N, d), s["W"][:F].float() * _spread(s["sw"][:half], F, d),
            s["W"][F:].float() * _spread(s["sw"][half:], F, d))


def _plain_blocks(s):
    N, d = s["x"].shape
    v = (s["x"].float() * _spread(s["sx"], N, d)) @ (s["W"].float() * _spread(s["sw"], s["d_out"], d)).t()
    v = _act(v if s["b"] is None else v + s["b"], s["act"])
    return (v if s["res"] is None else v + s["res"].float()).to(s["buf"].dtype)


def _plain_gated(s):
    x, Wg, Wu = _weights(s)
    return (_act(x @ Wg.t(), s["act"]) * (x @ Wu.t())).bfloat16()


def _plain_train(s):
    x, Wg, Wu = _weights(s)
    gate, up, dh = x @ Wg.t(), x @ Wu.t(), s["dh"].float()
    a = _act(gate, s["act"])
    dgate, dup = dh * up * _slope(gate, s["act"]), dh * a
    dx = dgate @ Wg + dup @ Wu
    dW = torch.cat([dgate.t() @ x, dup.t() @ x])
    return [(a * up).bfloat16(), dx.bfloat16(), dW.bfloat16()]


# ------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"bf16": 2, "fp32": 4, "e4m3": 1}
    N = case["N"]
    if case["op"] == "quantise":
        n = N * case["d"]
        return {"bytes": n * (size[case["dtype"]] + 1) + 4 * N * _blocks(case["d"]), "flops": 3 * n}
    d_in = case["d_in"]
    if case["op"] == "blocks":
        d_out = case["d_out"]
        return {"bytes": d_in * (N + d_out) + 4 * _blocks(d_in) * (N + _blocks(d_out)) + 4 * d_out * case["bias"]
                + size[case["y"]] * N * d_out * (1 + case["residual"]), "flops": 2 * N * d_in * d_out}
    d_ff = case["d_ff"]
    if case["op"] == "gated":
        scales = 4 * _blocks(d_in) * (N + 2 * _blocks(d_ff)) if case["dtype"] == "e4m3" else 0
        return {"bytes": size[case["dtype"]] * d_in * (N + 2 * d_ff) + scales + 2 * N * d_ff, "flops": 4 * N * d_in * d_ff}
    return {"bytes": 2 * (2 * N * d_in + 4 * d_in * d_ff + 2 * N * d_ff), "flops": 12 * N * d_in * d_ff}


# ------------------------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "quantise":
        v = s["x"].to(f)
        values, scales = torch.empty_like(v), []
        for c in range(0, case["d"], BLOCK):
            part = v[:, c:c + BLOCK]
            scales.append(torch.clamp(part.abs().max(dim=1).values, min=LOWEST_AMAX) / E4M3_MAX)
            values[:, c:c + BLOCK] = part / scales[-1][:, None]
        return values, torch.stack(scales, dim=1)

    def product(x, sx, W, sw):
        """x W^T, block of columns by block of columns, each with its scales."""
        if sx is None:
            return torch.matmul(x.to(f), W.to(f).T)
        total = torch.zeros(x.shape[0], W.shape[0], dtype=f, device=x.device)
        for b in range(sx.shape[1]):
            cols = slice(b * BLOCK, (b + 1) * BLOCK)
            rows = sw[:, b].to(f)[torch.arange(W.shape[0], device=x.device) // BLOCK]
            total += torch.matmul(x[:, cols].to(f), W[:, cols].to(f).T) * torch.outer(sx[:, b].to(f), rows)
        return total

    activation = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
                  "gelu": lambda v: 0.5 * v * torch.special.erfc(-v / math.sqrt(2)),
                  "gelu_tanh": lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}[case["act"]]
    if case["op"] == "blocks":
        y = product(s["x"], s["sx"], s["W"], s["sw"])
        y = activation(y + s["b"].to(f) if s["b"] is not None else y)
        return y + s["res"].to(f) if s["res"] is not None else y
    F = case["d_ff"]
    if case["op"] == "gated":
        half = _blocks(F)
        sg, su = (None, None) if s["sw"] is None else (s["sw"][:half], s["sw"][half:])
        return activation(product(s["x"], s["sx"], s["W"][:F], sg)) * product(s["x"], s["sx"], s["W"][F:], su)
    x, W = s["x"].to(f).requires_grad_(), s["W"].to(f).requires_grad_()
    gate, up = torch.matmul(x, W.T).split(F, dim=1)
    h = activation(gate) * up
    dx, dW = torch.autograd.grad(h, (x, W), s["dh"].to(f))
    return [h.detach(), dx, dW]
