"""The norm, the expert gate, the base product and the adapted projection against plain 64-bit
implementations of their formulas.

Tolerances, derived from the arithmetic (u = 2^-24, half a step of fp32; half a step of bf16 is 2^-8
and of e4m3 2^-4 of the value, 2^-10 below its normal range):
  * norm: every partial sum of squares passes at most 64 additions (up to 32 in a thread and 10 in the
    trees; about 70 + 10 for the longest row here, read element-wise by 1024 threads) of positive terms, so the sum
    is within 80 u + 1 u for the squares, its root within half of that; s, the root, the quotient
    and two products add 6 u.  Together under 64 u relative.
  * gate: expf is within 2 u (one ulp), its argument l - max (up to 40 here) within half a step of
    itself, 40 u of e; the sum, the quotient or 1 + e and its quotient, add 4 u: under 64 u of the
    score; renormalising and scaling over k <= 32 terms adds 35 u: under 128 u of the weight.  Choices closer than
    64 u (score + |bias|) may go either way; exact ties are made of equal inputs and have to go to
    the lower index.
  * product: each of the d_in additions loses at most a whole step (2 u) of a partial sum, itself
    at most S = sum |x w|: 2 u d_in S; tensor cores align products to the largest before adding,
    which is within the same whole step for each product; fp32 operands are cut into three bf16
    planes of which the products below 2^-21 |x w| (8 u) are left out: 8 u S.  The scales, the bias and the activation
    (whose slope is at most 1.13) add 16 u of what they handle; y rounds once.  Small
    integers, whose every partial sum is exact, have to come out bit for bit.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: U}
ACTS = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
        "gelu": lambda v: 0.5 * v * torch.erfc(-v / math.sqrt(2)),
        # (1 + tanh(u)) / 2 = sigmoid(2 u), without the cancellation at u < 0
        "gelu_tanh": lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}


@pytest.fixture(scope="module")
def m():
    from token_adapter_routing_gb300 import build
    build.build()
    import token_adapter_routing_gb300 as mod
    mod.load_library()
    return mod


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def within(got, want, tol):
    """Every element within tol; the message names the worst one."""
    over = (got.double() - want).abs() - tol
    assert not torch.isnan(over).any(), "NaN"
    i = int(over.argmax()) if over.numel() else 0
    assert over.numel() == 0 or over.flatten()[i] <= 0, \
        f"element {i}: got {got.double().flatten()[i].item()}, want {want.flatten()[i].item()}, tolerance " \
        f"{torch.as_tensor(tol, device='cuda').broadcast_to(want.shape).flatten()[i].item()}"


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def off_by_one(t):
    """A copy of t whose data starts one element into its buffer: contiguous, not 16-byte aligned."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


# ---------------------------------------------------------------------------------------- norm
def norm64(x, res, g, eps):
    s = x.double() + (res.double() if res is not None else 0.0)
    return s, s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps) * g.double()


def check_norm(x, res, g, eps, sum_out, out, out8, scale8):
    s, n = norm64(x, res, g, eps)
    tiny = 2.0 ** -140
    if sum_out is not None:
        within(sum_out, s, s.abs() * (HALF[x.dtype] + 2 * U) + tiny)
    if out is not None:
        within(out, n, n.abs() * (HALF[x.dtype] + 64 * U) + tiny)
    if out8 is not None:
        want = n.abs().amax(dim=1).clamp_min(2.0 ** -64) / 448
        within(scale8, want, want * 64 * U)
        q = n / want[:, None]
        within(out8.float(), q, q.abs() * (2.0 ** -4 + 256 * U) + 2.0 ** -10)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, d", [(1, 1), (1, 4096), (3, 7), (5, 8), (33, 64), (17, 100), (300, 512), (7, 2049), (129, 4096),
                                  (9, 6144), (4, 8191), (2, 16384), (3, 40000), (2, 70001), (5000, 96),
                                  (1300, 512), (1301, 4096), (2500, 1030), (1217, 2049), (1250, 5000), (1231, 8197), (1222, 16384),
                                  (4000, 263)])
@pytest.mark.parametrize("residual, fp8", [(False, False), (True, False), (True, True)])
def test_norm(m, dtype, N, d, residual, fp8):
    g = gen(N * 7 + d)
    x, w = (3 * randn(g, N, d)).to(dtype), (1 + 0.2 * randn(g, d)).to(dtype)
    res = randn(g, N, d).to(dtype) if residual else None
    out8 = torch.empty(N, d, dtype=FP8, device="cuda") if fp8 else None
    scale8 = torch.empty(N, device="cuda") if fp8 else None
    out = torch.empty_like(x) if (d % 2 or not fp8) else None
    got = m.molora_rmsnorm(x, w, 1e-5, residual=res, out=out, out8=out8, scale8=scale8)
    check_norm(x, res, w, 1e-5, *got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [37, 2500])
def test_norm_unaligned_and_in_place(m, dtype, N):
    g = gen(3)
    x, res, w = randn(g, N, 512).to(dtype), randn(g, N, 512).to(dtype), randn(g, 512).to(dtype)
    _, want, _, _ = m.molora_rmsnorm(x, w, 1e-6, residual=res)
    xo, ro = off_by_one(x), off_by_one(res)
    got_sum, got, _, _ = m.molora_rmsnorm(xo, off_by_one(w), 1e-6, residual=ro, sum_out=ro, out=xo)
    assert got is xo and got_sum is ro
    check_norm(x, res, w, 1e-6, ro, xo, None, None)
    x2, r2 = x.clone(), res.clone()
    m.molora_rmsnorm(x2, w, 1e-6, residual=r2, sum_out=r2, out=x2)
    assert torch.equal(x2, want)
    x3, r3 = x.clone(), res.clone()
    m.molora_rmsnorm(x3, w, 1e-6, residual=r3, sum_out=x3, out=r3)
    assert torch.equal(r3, want) and torch.equal(x3, r2)
    long = randn(g, 3, 70000).to(dtype)
    wl = randn(g, 70000).to(dtype)
    _, want, _, _ = m.molora_rmsnorm(long.clone(), wl)
    assert torch.equal(m.molora_rmsnorm(long, wl, out=long)[1], want)


def test_norm_extremes(m):
    """Zero rows, tiny rows, NaN and infinities stay in their rows; the rows behind the last one and the
    bytes behind the last element are left as they were."""
    g = gen(4)
    x = randn(g, 8, 192).to(BF)
    x[1] = 0
    x[2] = 1e-30
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    x[5] = 3e38
    w = torch.ones(192, dtype=BF, device="cuda")
    out = torch.full((10, 192), 7.0, dtype=BF, device="cuda")
    out8 = torch.full((10, 192), 7.0, device="cuda").to(FP8)
    scale8 = torch.full((10,), 7.0, device="cuda")
    m.molora_rmsnorm(x, w, 1e-6, out=out[:8], out8=out8[:8], scale8=scale8[:8])
    assert (out[8:] == 7).all() and (out8[8:].float() == 7).all() and (scale8[8:] == 7).all()
    assert (out[1] == 0).all() and (out8[1].float() == 0).all() and scale8[1] == 2.0 ** -64 / 448
    for row in (0, 1, 2, 6, 7):
        o8 = out8[row:row + 1]
        check_norm(x[row:row + 1], None, w, 1e-6, None, out[row:row + 1], o8, scale8[row:row + 1])
    assert torch.isnan(out[3]).all() and torch.isnan(scale8[3]) and torch.isnan(out8[3].float()).all()
    assert torch.isnan(out[4, 7]) and torch.isnan(scale8[4])
    assert (out[5] == 0).all() and scale8[5] == 2.0 ** -64 / 448  # the squares pass fp32's range


def test_norm_no_rows_and_streams(m):
    w = torch.ones(64, dtype=BF, device="cuda")
    s, o, o8, c8 = m.molora_rmsnorm(torch.empty(0, 64, dtype=BF, device="cuda"), w)
    assert o.shape == (0, 64) and s is None and o8 is None and c8 is None
    x = randn(gen(5), 2000, 64).to(BF)
    _, want, _, _ = m.molora_rmsnorm(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(x)
    m.molora_rmsnorm(x, w, out=got, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_norm_past_32_bit_offsets(m):
    N, d = 540000, 4096  # 2.2e9 elements
    x = torch.empty(N, d, dtype=BF, device="cuda")
    g = gen(6)
    x[:4], x[-4:] = randn(g, 4, d).to(BF), randn(g, 4, d).to(BF)
    x[4:-4] = 1
    w = torch.ones(d, dtype=BF, device="cuda")
    out8 = torch.empty(N, d, dtype=FP8, device="cuda")
    scale8 = torch.empty(N, device="cuda")
    out = m.molora_rmsnorm(x, w, out=x.clone(), out8=out8, scale8=scale8)[1]
    for part in (slice(0, 4), slice(N - 4, N)):
        check_norm(x[part], None, w, 1e-6, None, out[part], out8[part], scale8[part])


# ---------------------------------------------------------------------------------------- gate
def scores64(logits, score):
    l = logits.double()
    return torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)


def check_gate(logits, ids, w, k, score, bias, groups, keep, group_top, renorm, scale):
    """ids: distinct, descending and the largest of the kept groups, up to what 32 bits cannot tell
    apart; w: the chosen scores."""
    N, K = logits.shape
    s = scores64(logits, score)
    b = torch.zeros(K, device="cuda", dtype=torch.float64) if bias is None else bias.double()
    c = s + b
    tol = 64 * U * (s + b.abs()) + 2.0 ** -126
    ids = ids.long()
    assert ((ids >= 0) & (ids < K)).all()
    assert (torch.sort(ids, 1).values.diff(dim=1) > 0).all()
    if groups > 1:
        per = K // groups
        rank = c.view(N, groups, per).topk(group_top, dim=2).values.sum(2)
        rtol = 2 * group_top * tol.view(N, groups, per).amax(2).amax(1, keepdim=True)
        border = rank.topk(keep, dim=1).values[:, -1:]
        sure, maybe = rank > border + rtol, rank >= border - rtol
        used = torch.zeros(N, groups, dtype=torch.bool, device="cuda").scatter_(1, ids // per, True)
        assert (used <= maybe).all()
        open_group = (sure | used).repeat_interleave(per, dim=1)  # must have been open
    else:
        open_group = torch.ones(N, K, dtype=torch.bool, device="cuda")
    got, gtol = c.gather(1, ids), tol.gather(1, ids)
    assert (got[:, 1:] <= got[:, :-1] + gtol[:, 1:] + gtol[:, :-1]).all()
    rest = c.masked_fill(~open_group, -math.inf).scatter(1, ids, -math.inf)
    best, at = rest.max(dim=1)
    # an unchosen expert is no better than the last chosen one, nor the same with a lower index
    last = got[:, -1]
    assert (best <= last + gtol[:, -1] + tol.gather(1, at[:, None])[:, 0]).all()
    want = s.gather(1, ids)
    if renorm:
        want = want / want.sum(1, keepdim=True)
    within(w, want * scale, (want * scale).abs() * 128 * U + 2.0 ** -126)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, K, k, score, bias, groups, keep, top", [
    (1, 1, 1, "softmax", False, 1, 1, 1), (1, 64, 2, "softmax", False, 1, 1, 1), (33, 4, 4, "sigmoid", True, 1, 1, 1),
    (257, 60, 6, "softmax", True, 1, 1, 1), (1000, 256, 8, "sigmoid", True, 8, 4, 2), (63, 512, 32, "softmax", True, 1, 1, 1),
    (100, 512, 8, "sigmoid", False, 32, 3, 2), (77, 66, 5, "softmax", False, 6, 2, 1), (129, 30, 3, "sigmoid", False, 5, 5, 1),
    (64, 255, 7, "softmax", True, 3, 1, 2), (200, 33, 33 - 1, "sigmoid", False, 1, 1, 1), (50, 16, 2, "softmax", True, 8, 1, 2),
    (513, 128, 6, "softmax", False, 1, 1, 1), (90, 48, 4, "softmax", True, 16, 4, 1), (40, 250, 9, "sigmoid", True, 25, 20, 2),
    (70, 32, 5, "softmax", True, 32, 9, 1), (45, 64, 6, "sigmoid", True, 2, 1, 2), (91, 128, 32, "softmax", True, 4, 3, 2),
    (37, 512, 8, "softmax", True, 16, 5, 2), (21, 256, 12, "softmax", False, 8, 2, 1)])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate(m, dtype, N, K, k, score, bias, groups, keep, top, renorm):
    g = gen(N + K)
    logits = (2 * randn(g, N, K)).to(dtype)
    b = 0.1 * randn(g, K) if bias else None
    e = err_word()
    ids, w = m.molora_gate_topk(logits, k, score=score, bias=b, groups=groups, keep_groups=keep, group_top=top,
                                renormalise=renorm, scale=2.5, err_word=e)
    check_gate(logits, ids, w, k, score, b, groups, keep, top, renorm, 2.5)
    assert e.item() == 0
    again = m.molora_gate_topk(off_by_one(logits), k, score=score, bias=b, groups=groups, keep_groups=keep, group_top=top,
                               renormalise=renorm, scale=2.5)
    assert torch.equal(ids, again[0]) and torch.equal(w, again[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("K, groups, top", [(16, 1, 1), (60, 1, 1), (256, 8, 2), (64, 4, 1), (500, 1, 1),
                                            (512, 4, 2), (96, 4, 2)])
def test_gate_ties_go_to_the_lower_index(m, score, K, groups, top):
    """Logits of three values only: among equal experts, and equal groups, the lower index comes first."""
    g = gen(K)
    N, k, keep = 200, 4, max(1, groups // 2)
    logits = torch.randint(0, 3, (N, K), generator=g, device="cuda").float()
    ids, _ = m.molora_gate_topk(logits, k, score=score, groups=groups, keep_groups=keep, group_top=top)
    c = logits.double() if groups == 1 or top == 1 else torch.sigmoid(logits.double()) if score == "sigmoid" else logits.double().exp()
    if groups > 1:
        rank = c.view(N, groups, -1).topk(top, dim=2).values.sum(2)
        kept = torch.argsort(-rank, dim=1, stable=True)[:, :keep]
        mask = torch.zeros(N, groups, device="cuda", dtype=torch.bool).scatter_(1, kept, True)
        c = c.masked_fill(~mask.repeat_interleave(K // groups, dim=1), -math.inf)
    assert torch.equal(ids.long(), torch.argsort(-c, dim=1, stable=True)[:, :k])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups, top", [(1, 1), (4, 1), (4, 2)])
def test_gate_masked_experts(m, score, groups, top):
    g = gen(9)
    N, K, k = 6, 32, 4
    logits = randn(g, N, K)
    logits[0] = -math.inf                       # nothing left
    logits[1, 3:] = -math.inf                   # three experts left, all in group 0
    logits[2, 5] = math.nan
    logits[3, 7] = math.inf
    logits[4] = torch.finfo(F32).min            # the type's lowest value is a logit like any other
    logits[5, ::2] = -math.inf
    e = err_word()
    ids, w = m.molora_gate_topk(logits, k, score=score, groups=groups, keep_groups=groups, group_top=top, err_word=e)
    assert (ids[0] == -1).all() and (w[0] == 0).all()
    assert sorted(ids[1, :3].tolist()) == [0, 1, 2] and ids[1, 3] == -1 and w[1, 3] == 0
    assert abs(w[1].sum().item() - 1) < 8 * U
    assert 5 not in ids[2].tolist() and (ids[2] >= 0).all()
    assert ids[3, 0] == 7 and w[3, 0] > 0
    assert ids[4].tolist() == [0, 1, 2, 3]
    assert (ids[5] % 2 == 1).all()
    assert not torch.isnan(w).any()
    assert e.item() == m.DEV_BAD_LOGIT
    # rows of ids feed the dispatch: slots of -1 are left out
    counts, offsets, perm = m.molora_dispatch(ids, K, err_word=e)
    assert counts.sum().item() == (ids >= 0).sum().item()


def test_gate_bias_extremes(m):
    logits = torch.zeros(2, 8, device="cuda")
    b = torch.zeros(8, device="cuda")
    b[0], b[1], b[2] = -math.inf, math.inf, math.nan
    e = err_word()
    ids, w = m.molora_gate_topk(logits, 6, bias=b, err_word=e)
    assert ids.tolist() == [[1, 3, 4, 5, 6, 7]] * 2 and e.item() == m.DEV_BAD_LOGIT
    within(w, torch.full_like(w, 1 / 6).double(), 8 * U)


def test_gate_rows_behind_and_no_rows(m):
    ids = torch.full((9, 2), 77, dtype=torch.int32, device="cuda")
    w = torch.full((9, 2), 7.0, device="cuda")
    m.molora_gate_topk(randn(gen(1), 7, 40), 2, ids=ids[:7], w=w[:7])
    assert (ids[7:] == 77).all() and (w[7:] == 7).all() and (ids[:7] < 40).all()
    ids, w = m.molora_gate_topk(torch.empty(0, 40, device="cuda"), 2)
    assert ids.shape == (0, 2)


def test_gate_past_32_bit_offsets(m):
    N, K = 4_200_000, 512
    logits = torch.zeros(N, K, dtype=BF, device="cuda")
    logits[:, 17] = 1
    logits[-3:] = randn(gen(2), 3, K).to(BF)
    ids, w = m.molora_gate_topk(logits, 2, score="sigmoid")
    assert (ids[:-3, 0] == 17).all() and (ids[:-3, 1] == 0).all()
    check_gate(logits[-3:], ids[-3:], w[-3:], 2, "sigmoid", None, 1, 1, 1, True, 1.0)


# ---------------------------------------------------------------------------------------- product
def quantised(v):
    scale = v.abs().amax(dim=1).clamp_min(2.0 ** -64) / 448
    return (v / scale[:, None]).clamp(-448, 448).to(FP8), scale


def linear_inputs(g, N, d_in, d_out, dtype):
    x, W = randn(g, N, d_in), randn(g, d_out, d_in) / math.sqrt(d_in)
    if dtype == FP8:
        (x, sx), (W, sw) = quantised(x), quantised(W)
        return x, W, sx, sw
    return x.to(dtype), W.to(dtype), None, None


def check_linear(y, x, W, sx, sw, bias, act, res):
    xd, wd = x.double(), W.double()
    scale = torch.ones(1, 1, device="cuda", dtype=torch.float64) if sx is None else sx.double()[:, None] * sw.double()[None]
    v, S = xd @ wd.T * scale, xd.abs() @ wd.abs().T * scale
    tol = S * (2 * U * (x.shape[1] + 16)) + S * (8 * U if x.dtype == F32 else 0)
    if bias is not None:
        v, tol = v + bias.double(), tol + 16 * U * bias.double().abs()
    a = ACTS[act](v)
    tol = 1.13 * tol + 16 * U * (v.abs() if act != "none" else 0)
    if res is not None:
        a, tol = a + res.double(), tol + 2 * U * res.double().abs()
    within(y, a, tol + a.abs() * (HALF[y.dtype] + 2 * U) + 2.0 ** -120)


@pytest.mark.parametrize("act", sorted(ACTS))
def test_linear_activation_curves(m, act):
    """act over its whole range, the sums exact (d_in = 1, W = 1): a power and a reciprocal are good to 2^-22
    and 2^-23, an exponent's rounding costs 2 U of it; below the normal numbers they are 0.  So are the lower two
    of an operand's three bf16 parts where they are below 2^-126, which is less than 2^-125 together.  v / (1 + e)
    takes the sum's rounding (U), the reciprocal (2^-23 = 2 U) and the product's (U): under 5 U of the result."""
    v = torch.cat([s * torch.logspace(-38, 38, 3001, device="cuda") for s in (1, -1)] +
                  [torch.linspace(-16, 16, 8001, device="cuda"), torch.zeros(1, device="cuda")])
    y = m.molora_linear(v[:, None], torch.ones(1, 1, device="cuda"), act=act, out_dtype=F32)[:, 0]
    d = v.double()
    want = ACTS[act](d)
    want[(d < -100) & (act != "none")] = 0
    exponent = {"silu": d.abs(), "gelu": d * d, "gelu_tanh": 1.6 * d.abs() + 0.072 * d.abs() ** 3}.get(act, 0 * d)
    tail = want - d.clamp_min(0) if act != "none" else 0 * d   # what the power makes
    within(y, want, 5 * U * want.abs() + tail.abs() * (2.0 ** -20 + 4 * U * exponent) + d.abs().clamp(1, 100) * 2.0 ** -125)
    odd = torch.tensor([[math.inf], [math.nan], [-math.inf]], device="cuda")
    y = m.molora_linear(odd, torch.ones(1, 1, device="cuda"), act=act, out_dtype=F32)[:, 0].tolist()
    assert y[0] == math.inf and math.isnan(y[1])
    if act in ("relu", "gelu"):
        assert y[2] == 0


SIZES = [(1, 64, 64), (1, 4096, 1000), (2, 128, 7), (3, 33, 5), (7, 200, 257), (8, 2048, 512), (16, 512, 129), (17, 640, 384),
         (31, 1031, 517), (33, 4096, 96), (64, 96, 64), (65, 256, 1024), (127, 512, 260), (128, 64, 128), (129, 1024, 256),
         (200, 72, 200), (257, 2048, 320), (300, 24, 24), (513, 1, 1), (700, 136, 1032), (1024, 512, 768),
         (2500, 272, 2056), (3001, 1024, 1100), (4097, 64, 1333), (20000, 128, 160),
         (1, 260, 2100), (1, 1031, 517), (1, 4096, 257), (1, 8, 3), (2, 512, 2305), (4, 516, 2051), (3, 128, 4097), (4, 4100, 65),
         (1, 1024, 33), (2, 1024, 1000), (4, 1024, 513), (3, 512, 2048), (2, 333, 2049), (3, 1031, 34), (4, 77, 2050)]


@pytest.mark.parametrize("N, d_in, d_out", SIZES)
@pytest.mark.parametrize("dtype", [BF, FP8, F32])
@pytest.mark.parametrize("y_dtype, bias, act, residual", [(F32, False, "none", False), (BF, True, "silu", True),
                                                          (F32, True, "gelu", True), (BF, False, "gelu_tanh", False),
                                                          (F32, True, "relu", False)])
def test_linear(m, N, d_in, d_out, dtype, y_dtype, bias, act, residual):
    g = gen(N + d_in + d_out)
    x, W, sx, sw = linear_inputs(g, N, d_in, d_out, dtype)
    b = randn(g, d_out) if bias else None
    res = randn(g, N, d_out).to(y_dtype) if residual else None
    buf = torch.full((N + 3, d_out), 7.0, dtype=y_dtype, device="cuda")
    e = err_word()
    y = m.molora_linear(x, W, y=buf[:N], x_scale=sx, w_scale=sw, bias=b, act=act, residual=res, err_word=e)
    assert e.item() == 0
    check_linear(y, x, W, sx, sw, b, act, res)
    assert (buf[N:] == 7).all()


@pytest.mark.parametrize("N, d_in, d_out", [(1, 512, 512), (5, 64, 40), (40, 1024, 136), (130, 320, 264), (600, 4096, 512), (2, 333, 31),
                                            (2900, 160, 2100), (2600, 512, 2052), (5000, 96, 1031)])
@pytest.mark.parametrize("dtype", [BF, FP8, F32])
def test_linear_integers_are_exact(m, N, d_in, d_out, dtype):
    g = gen(d_in)
    x = torch.randint(-4, 5, (N, d_in), generator=g, device="cuda").float()
    W = torch.randint(-4, 5, (d_out, d_in), generator=g, device="cuda").float()
    res = torch.randint(-100, 100, (N, d_out), generator=g, device="cuda").float()
    scales = {}
    if dtype == FP8:
        scales = {"x_scale": torch.ones(N, device="cuda"), "w_scale": 2.0 * torch.ones(d_out, device="cuda")}
    y = m.molora_linear(x.to(dtype), W.to(dtype), residual=res, **scales)
    want = (x.double() @ W.double().T) * (2 if scales else 1) + res.double()
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("dtype", [BF, FP8, F32])
@pytest.mark.parametrize("N, d_in, d_out", [(4, 256, 96), (150, 256, 192), (4000, 64, 1024)])
def test_linear_unaligned_and_in_place(m, dtype, N, d_in, d_out):
    g = gen(11)
    x, W, sx, sw = linear_inputs(g, N, d_in, d_out, dtype)
    res, b = randn(g, N, d_out), randn(g, d_out)
    y = off_by_one(res)
    m.molora_linear(off_by_one(x), off_by_one(W), y=y, x_scale=sx, w_scale=sw, bias=off_by_one(b), residual=y)
    check_linear(y, x, W, sx, sw, b, "none", res)
    y = res.clone()
    m.molora_linear(x, W, y=y, x_scale=sx, w_scale=sw, bias=b, residual=y)
    check_linear(y, x, W, sx, sw, b, "none", res)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, d_in, d_out", [(3, 256, 64), (140, 256, 64), (5, 255, 33), (3000, 256, 1024), (150, 1023, 70)])
def test_linear_nan_and_infinity_stay_in_their_rows(m, dtype, N, d_in, d_out):
    g = gen(12)
    x, W, _, _ = linear_inputs(g, N, d_in, d_out, dtype)
    x[1, 3], x[2, 4] = math.nan, math.inf
    y = m.molora_linear(x, W)
    assert torch.isnan(y[1]).all()
    assert torch.equal(y[2], torch.where(W[:, 4] > 0, math.inf, -math.inf))
    rest = [0] + list(range(3, N))
    check_linear(y[rest], x[rest], W, None, None, None, "none", None)
    # and an infinite weight in its column
    x, W, _, _ = linear_inputs(g, N, d_in, d_out, dtype)
    W[5, 7] = -math.inf
    y = m.molora_linear(x, W, act="relu")
    assert torch.equal(y[:, 5], torch.where(x[:, 7] > 0, 0.0, math.inf))
    cols = [i for i in range(d_out) if i != 5]
    check_linear(y[:, cols], x, W[cols], None, None, None, "relu", None)


def test_linear_fp32_range(m):
    """Values next to fp32's largest and below its normal range are cut into planes without loss."""
    g = gen(15)
    N, d_in, d_out = 20, 96, 40
    x, W = torch.zeros(N, d_in, device="cuda"), torch.zeros(d_out, d_in, device="cuda")
    x[:, 0], W[:, 0] = torch.finfo(F32).max, randn(g, d_out).sign()
    assert torch.equal(m.molora_linear(x, W), x[:, :1] * W[:, 0])
    x[:, 0], W[:, 0] = 2.0 ** -100 * randn(g, N), 2.0 ** 90 * randn(g, d_out)
    y = m.molora_linear(x, W).double()
    want = x[:, :1].double() * W[:, 0].double()
    within(y, want, want.abs() * 8 * U)


def test_linear_no_rows(m):
    W = torch.ones(8, 64, dtype=BF, device="cuda")
    assert m.molora_linear(torch.empty(0, 64, dtype=BF, device="cuda"), W).shape == (0, 8)


@pytest.mark.parametrize("dtype, d_in", [(BF, 64), (F32, 16)])
def test_linear_past_32_bit_offsets(m, dtype, d_in):
    N, d_out = 2_200_000, 1024
    g = gen(13)
    x, W, _, _ = linear_inputs(g, N, d_in, d_out, dtype)
    y = m.molora_linear(x, W, out_dtype=BF)
    for part in (slice(0, 5), slice(N - 5, N)):
        check_linear(y[part], x[part], W, None, None, None, "none", None)


@pytest.mark.parametrize("dtype", [BF, FP8, F32])
def test_linear_results_repeat(m, dtype):
    for N in (1, 20, 300):
        g = gen(14)
        x, W, sx, sw = linear_inputs(g, N, 2048, 512, dtype)
        first = m.molora_linear(x, W, x_scale=sx, w_scale=sw)
        for _ in range(5):
            assert torch.equal(first, m.molora_linear(x, W, x_scale=sx, w_scale=sw))


# ---------------------------------------------------------------------------------------- together
def layer(g, N, d_in, d_out, K, r, k, fp8):
    x, res = randn(g, N, d_in).to(BF), randn(g, N, d_in).to(BF)
    nw = (1 + 0.1 * randn(g, d_in)).to(BF)
    W, sw = quantised(randn(g, d_out, d_in) / math.sqrt(d_in)) if fp8 else ((randn(g, d_out, d_in) / math.sqrt(d_in)).to(BF), None)
    A, B = (randn(g, K, d_in, r) / math.sqrt(d_in)).to(BF), (randn(g, K, r, d_out) / math.sqrt(r)).to(BF)
    Wg, b = (randn(g, K, d_in) / math.sqrt(d_in)).to(BF), randn(g, d_out)
    return x, res, nw, W, sw, A, B, Wg, b


@pytest.mark.parametrize("y_dtype", [F32, BF])
@pytest.mark.parametrize("N, d_in, d_out, K, r, k, fp8", [
    (1, 512, 512, 4, 16, 1, False), (16, 512, 640, 8, 16, 2, True), (300, 256, 384, 4, 16, 2, False),
    (1500, 512, 512, 8, 64, 2, True), (2100, 256, 256, 4, 16, 1, False), (33, 520, 264, 3, 8, 2, False),
    # the product takes the update along: K*r of one, part of one and several K blocks, widths of every tile
    (2600, 512, 2048, 4, 16, 2, False), (4000, 256, 1544, 2, 16, 1, False), (2300, 320, 2120, 3, 32, 2, False),
    (5000, 128, 1024, 8, 64, 3, False), (20000, 64, 160, 4, 32, 2, False),
    (2305, 1088, 1920, 7, 64, 2, False), (2900, 64, 2048, 13, 32, 1, False),
    (2600, 512, 2048, 4, 16, 2, True), (300, 1088, 392, 3, 32, 2, True), (5000, 128, 1024, 8, 64, 3, True)])
def test_adapted_layer(m, y_dtype, N, d_in, d_out, K, r, k, fp8):
    """Norm -> linear gate -> gate -> dispatch -> the adapted projection, as a layer runs them, against
    the formulas in 64 bits on what each call reads; and the one call against the three it chains."""
    g = gen(N)
    x, res, nw, W, sw, A, B, Wg, b = layer(g, N, d_in, d_out, K, r, k, fp8)
    e = err_word()
    _, h0, _, _ = m.molora_rmsnorm(x, nw, 1e-6, residual=res)
    logits = m.molora_linear(h0, Wg, err_word=e)
    ids, w = m.molora_gate_topk(logits, k, bias=None, err_word=e)
    counts, offsets, perm = m.molora_dispatch(ids, K, err_word=e)
    y = torch.empty(N, d_out, dtype=y_dtype, device="cuda")
    _, s, h, h8, scale8 = m.molora_norm_linear_lora_apply(
        x, nw, 1e-6, W, A, B, ids, y, 2.0, w=w, counts=counts, offsets=offsets, perm=perm, residual=res, w_scale=sw, bias=b,
        err_word=e)
    assert e.item() == 0
    check_norm(x, res, nw, 1e-6, s, h, h8, scale8)
    assert torch.equal(h, h0)
    # 64 bits, from the rows as stored
    base = (h8.double() * scale8.double()[:, None]) @ (W.double() * sw.double()[:, None]).T if fp8 else h.double() @ W.double().T
    hd = h.double()
    update = torch.zeros_like(base)
    for a in range(K):
        wa = (w.double() * (ids == a)).sum(1, keepdim=True)
        update += 2.0 * wa * ((hd @ A[a].double()) @ B[a].double())
    want = base + b.double() + update
    rms = want.pow(2).mean().sqrt().item()
    # the apply's own bar (2e-4 rms in fp32); bf16 y rounds the base, and each slot once more
    mag = base.abs() + b.double().abs() + update.abs() + want.abs()
    within(y, want, 2e-4 * rms + (0 if y_dtype == F32 else (k + 1) * 2.0 ** -8 * (mag + rms)))
    # the same three calls one by one
    y2 = m.molora_linear(h8 if fp8 else h, W, x_scale=scale8, w_scale=sw, bias=b, out_dtype=y_dtype)
    m.molora_lora_apply(h, A, B, ids, y2, 2.0, w=w, counts=counts, offsets=offsets, perm=perm)
    # the grouped apply adds a token's k > 1 slots in no fixed order; bf16 y takes it where fp32 y takes
    # the stacked pair
    path = m.molora_select_path(BF, N, d_in, d_out, K, r, k)
    if N > 256 and d_in % 64 == 0 and r >= 16 and K * r <= 512:
        # the product has taken the update along, whose shrink is held in two bf16 terms (2^-17)
        within(y, y2.double(), 4e-4 * rms if y_dtype == F32 else 2 * (k + 1) * 2.0 ** -8 * (mag + rms))
    elif k == 1 or path in ("scalar", "dense") or (path == "stacked" and y_dtype == F32):
        assert torch.equal(y, y2)
    else:
        within(y, y2.double(), 4e-4 * rms if y_dtype == F32 else 2 * (k + 1) * 2.0 ** -8 * (mag + rms))


@pytest.mark.parametrize("N", [48, 400])
def test_layer_captured_and_replayed(m, N):
    """The chain in a CUDA graph, replayed on new inputs, equals the eager calls; two graphs alive
    at once do not disturb one another."""
    d, K, r, k = 512, 8, 16, 2
    graphs = []
    for seed, fp8 in ((21, True), (22, False)):
        tensors = layer(gen(seed), N, d, d, K, r, k, fp8)
        x = tensors[0]

        def step(tensors=tensors):
            x, res, nw, W, sw, A, B, Wg, b = tensors
            _, h, _, _ = m.molora_rmsnorm(x, nw, 1e-6, residual=res)
            ids, w = m.molora_gate_topk(m.molora_linear(h, Wg), k, score="sigmoid")
            y = torch.empty(N, d, device="cuda")
            m.molora_norm_linear_lora_apply(x, nw, 1e-6, W, A, B, ids, y, 2.0, w=w, residual=res, w_scale=sw, bias=b)
            return ids, w, y
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out, x, step))
    for n in range(3):
        for graph, out, x, step in graphs:
            x.copy_(randn(gen(100 + n), N, d))
        for graph, _, _, _ in graphs:
            graph.replay()
        for _, out, _, step in graphs:
            want = step()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N", [5, 300])
def test_fp32_layer(m, N, fp8):
    """Hidden states and adapters in fp32, base weights in fp32 or e4m3."""
    g = gen(41 + N)
    d_in, d_out, K, r, k = 192, 160, 3, 8, 2
    x, nw, A, B = randn(g, N, d_in), 1 + 0.1 * randn(g, d_in), randn(g, K, d_in, r) / math.sqrt(d_in), randn(g, K, r, d_out)
    W, sw = randn(g, d_out, d_in) / math.sqrt(d_in), None
    if fp8:
        W, sw = quantised(W)
    ids, w = m.molora_gate_topk(randn(g, N, K), k)
    buf = torch.full((N + 2, d_out), 7.0, device="cuda")
    y, s, h, h8, scale8 = m.molora_norm_linear_lora_apply(x, nw, 1e-6, W, A, B, ids, buf[:N], 2.0, w=w, w_scale=sw)
    assert s is None and (buf[N:] == 7).all() and (h8 is not None) == fp8
    check_norm(x, None, nw, 1e-6, None, h, h8, scale8)
    base = (h8.double() * scale8.double()[:, None]) @ (W.double() * sw.double()[:, None]).T if fp8 else h.double() @ W.double().T
    for a in range(K):
        base += 2.0 * (w.double() * (ids == a)).sum(1, keepdim=True) * ((h.double() @ A[a].double()) @ B[a].double())
    within(y, base, 2e-4 * base.pow(2).mean().sqrt().item())


@pytest.mark.parametrize("N", [20, 300])
def test_layer_skips_slots_without_an_adapter(m, N):
    """Slots of -1 (a token whose experts ran out) are skipped and reported; the others are applied."""
    g = gen(51)
    x, _, nw, W, _, A, B, _, _ = layer(g, N, 256, 192, 4, 16, 2, False)
    ids = torch.randint(0, 4, (N, 2), generator=g, device="cuda", dtype=torch.int32)
    ids[:, 1] = torch.where(torch.arange(N, device="cuda") % 3 == 0, -1, (ids[:, 0] + 1) % 4)
    w = torch.rand(N, 2, generator=g, device="cuda")
    e = err_word()
    y = torch.empty(N, 192, device="cuda")
    _, _, h, _, _ = m.molora_norm_linear_lora_apply(x, nw, 1e-6, W, A, B, ids, y, 2.0, w=w, err_word=e)
    assert e.item() == m.DEV_BAD_ADAPTER_ID
    want = h.double() @ W.double().T
    for a in range(4):
        want += 2.0 * (w.double() * (ids == a)).sum(1, keepdim=True) * ((h.double() @ A[a].double()) @ B[a].double())
    within(y, want, 2e-4 * want.pow(2).mean().sqrt().item())


@pytest.mark.parametrize("y_dtype", [BF, F32])
def test_buffers_of_a_call_on_another_stream(m, y_dtype):
    """What a call on a given stream makes for itself stays its own until that stream is done: buffers
    made and dropped on the current stream meanwhile get other memory."""
    g = gen(37)
    N, d, K, r = 600, 512, 4, 16
    x, _, nw, W, sw, A, B, Wg, _ = layer(g, N, d, d, K, r, 2, True)
    ids, w = m.molora_gate_topk(m.molora_linear(x, Wg), 2)
    want = torch.empty(N, d, device="cuda", dtype=y_dtype)
    m.molora_norm_linear_lora_apply(x, nw, 1e-6, W, A, B, ids, want, 2.0, w=w, w_scale=sw)
    y = torch.empty_like(want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(50_000_000)           # the call's kernels wait for this
    m.molora_norm_linear_lora_apply(x, nw, 1e-6, W, A, B, ids, y, 2.0, w=w, w_scale=sw, stream=st)
    h = m.molora_rmsnorm(x, nw, stream=st)[1]
    logits = m.molora_linear(h, Wg, stream=st)
    others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (N * d * 2, N * d, N * 4, N * K * r * 4) * 4]
    st.synchronize()
    assert torch.equal(y, want)
    assert torch.equal(h, m.molora_rmsnorm(x, nw)[1])
    assert torch.equal(logits, m.molora_linear(h, Wg))
    assert all((o == 255).all() for o in others)


def test_two_streams_at_once(m):
    g = gen(31)
    x, W, _, _ = linear_inputs(g, 300, 1024, 512, BF)
    nw = torch.ones(1024, dtype=BF, device="cuda")
    want = m.molora_linear(m.molora_rmsnorm(x, nw)[1], W)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(m.molora_linear(m.molora_rmsnorm(x, nw)[1], W))
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o, want)
