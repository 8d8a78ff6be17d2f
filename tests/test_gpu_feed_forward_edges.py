"""The feed-forward kernels at the ends of their ranges: activations over every gate and beside values that have none, sums of
many terms, quotients to the last bit.

Tolerances (u = 2^-24, half a step of fp32): an activation's exponent z, 126 at most before its power is flushed, is made with up to
four roundings of it, so its power is off by 126 ln 2 * 4 u = 350 u; the power itself (4 u), the sum, the products and the
reciprocal add fewer than 30: 384 u of the result.  Below 2^-126 powers are 0, where v / (1 + 2^z) is below 2^-119."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: U}
ACTS = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
        "gelu": lambda v: 0.5 * v * torch.erfc(-v / math.sqrt(2)),
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
    over = (got.double() - want).abs() - tol
    assert not torch.isnan(over).any(), "NaN"
    i = int(over.argmax())
    assert over.flatten()[i] <= 0, f"element {i}: got {got.double().flatten()[i].item()}, want {want.flatten()[i].item()}"


# ---------------------------------------------------------------------------------------- activations
@pytest.mark.parametrize("y_dtype", [F32, BF])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("N", [1, 32, 512])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activations_over_the_whole_range(m, act, N, odd, y_dtype):
    """act(bias) of every finite bf16 value through the block-scaled product of zeros (few tokens, many, rows that start
    anywhere), in an order that puts values of all sizes beside one another."""
    v = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(BF).float()
    v = v[torch.isfinite(v)]
    v = v[(v == 0) | (v.abs() >= 2.0 ** -118)]
    v = torch.cat([v, v[torch.randperm(v.numel(), generator=gen(1), device="cuda")]])  # neighbours in size, then any
    v = v[:v.numel() // 8 * 8 - odd]
    x, W = torch.zeros(N, 16, device="cuda").to(FP8), torch.zeros(v.numel(), 16, device="cuda").to(FP8)
    one = torch.ones(N, 1, device="cuda"), torch.ones(-(-v.numel() // 128), 1, device="cuda")
    y = m.molora_linear_blocks(x, one[0], W, one[1], bias=v.clone(), act=act, out_dtype=y_dtype)
    want = ACTS[act](v.double())
    within(y, want.expand(N, -1), want.abs() * (384 * U + HALF[y_dtype]) + 2.0 ** -118)


@pytest.mark.parametrize("N", [32, 4096])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_gates_over_the_whole_range(m, act, N):
    """Every e4m3 value times scales of all sizes as the gate, each exact, through few tokens' kernel and many's."""
    w = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).view(FP8).float()
    w = w[torch.isfinite(w)]
    w = torch.cat([w, w[torch.randperm(w.numel(), generator=gen(2), device="cuda")]])
    w = w.repeat(4)[:2032]
    F = w.numel()
    x, W = torch.zeros(N, 16, device="cuda"), torch.zeros(2 * F, 16, device="cuda")
    x[:, 0], W[:F, 0], W[F:, 0] = 1, w, 1
    sx = torch.exp2(torch.linspace(-24, 8, N, device="cuda"))
    sw = torch.ones(2 * -(-F // 128), 1, device="cuda")
    h = m.molora_gated_linear(x.to(FP8), W.to(FP8), act=act, x_scale=sx[:, None].contiguous(), w_scale=sw)
    gate = sx.double()[:, None] * w.double()   # (rounds once to fp32, and act' is 1.13 at most, or what moves |z| ln 2 <= 88 by u)
    want = ACTS[act](gate) * sx.double()[:, None]
    within(h, want, want.abs() * (512 * U + HALF[BF]) + 2.0 ** -118 * sx.double()[:, None] + 2.0 ** -126)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("N", [8, 512])
def test_activations_beside_nan_and_infinity(m, act, N):
    """A NaN or an infinity in one column leaves those beside it within their own tolerance."""
    g = gen(N)
    v = 40 * randn(g, 4096)
    v[1::7], v[3::11], v[5::13], v[8::17] = math.nan, math.inf, -math.inf, -3e38
    x, W = torch.zeros(N, 16, device="cuda").to(FP8), torch.zeros(4096, 16, device="cuda").to(FP8)
    y = m.molora_linear_blocks(x, torch.ones(N, 1, device="cuda"), W, torch.ones(32, 1, device="cuda"), bias=v, act=act)
    assert torch.isnan(y[:, torch.isnan(v)]).all() and (y[:, v == math.inf] == math.inf).all()
    want = ACTS[act](v.double())[torch.isfinite(v)]
    within(y[:, torch.isfinite(v)], want.expand(N, -1), want.abs() * 385 * U + 2.0 ** -118)


# ---------------------------------------------------------------------------------------- long sums
def positive(g, rows, cols, by_row=False):
    """Values from 1/2 to 1, of columns (or rows) of different sizes: sums of them that fall anywhere between two bf16 values."""
    s = torch.exp2(torch.rand((rows, 1) if by_row else (1, cols), generator=g, device="cuda"))
    return ((0.5 + 0.5 * torch.rand(rows, cols, generator=g, device="cuda")) * s).to(BF)


def drift(got, want):
    """How far the outputs are off together, and what may be: 2^-15, a 128th of what bf16's rounding may do to each, for what a
    tensor core's additions cut; the mean of that rounding (2^-8 at most of an output, 2^-8 / sqrt(3) at most on the root mean
    square, either way: six deviations); 2^-20 for fp32's few additions.  An addition that cuts to fp32 loses half a step, 2^-25 of
    the sum at least, on the mean: a single chain of n MMAs of 16 terms is 2^-25 sum_j j / n = 2^-26 n short at least, 1.2e-4 for
    2^17 terms and 2.4e-4 for 2^18."""
    off = ((got.double() - want) / want).mean().abs().item()
    return off, 2.0 ** -15 + 6 * 2.0 ** -8 / math.sqrt(3 * want.numel()) + 2.0 ** -20


def test_many_tokens_dw_does_not_drift(m):
    """dW's sums run over the tokens, however many there are."""
    g, N, d, F = gen(70), (1 << 18) + 77, 512, 256
    x, W, dh = positive(g, N, d), positive(g, 2 * F, d), positive(g, N, F)
    dx, dW, dproj = m.molora_gated_linear_backward(x, W, dh, act="none", want_dx=False)
    want = torch.zeros(2 * F, d, dtype=torch.float64, device="cuda")
    for t in range(0, N, 1 << 16):
        want += dproj[t:t + (1 << 16)].view(-1, 2 * F).double().T @ x[t:t + (1 << 16)].double()
    off, most = drift(dW, want)
    assert off <= most, (off, most)


def test_wide_blocks_dx_does_not_drift(m):
    """dx's sums run over both projections' columns."""
    g, N, d, F = gen(71), 8192, 512, 1 << 16
    x, W, dh = (positive(g, N, d) / 512).to(BF), positive(g, 2 * F, d), positive(g, N, F, by_row=True)
    dx, _, dproj = m.molora_gated_linear_backward(x, W, dh, act="none", want_dW=False)
    want = torch.zeros(N, d, dtype=torch.float64, device="cuda")
    for f in range(0, 2 * F, 1 << 14):
        want += dproj.view(N, 2 * F)[:, f:f + (1 << 14)].double() @ W[f:f + (1 << 14)].double()
    off, most = drift(dx, want)
    assert off <= most, (off, most)


@pytest.mark.parametrize("N, d, F", [(8192, 264, 130), (8193, 264, 130), (40000, 136, 65), (300, 520, 20000), (3000, 1032, 4100)])
def test_gradients_of_long_sums(m, N, d, F):
    """Sums of one chain of K blocks, one more, several, and of dx's and dW's different numbers of them, every output against the
    64-bit sums of the same dproj (n additions each lose at most a step of a partial sum: 2 u n S), and the same bits again."""
    g = gen(N + F)
    x, W, dh = randn(g, N, d).to(BF), (randn(g, 2 * F, d) / math.sqrt(d)).to(BF), randn(g, N, F).to(BF)
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dW, dproj = m.molora_gated_linear_backward(x, W, dh, err_word=e)
    assert e.item() == 0
    dp = torch.cat([dproj[:, 0, :F], dproj[:, 1, :F]], dim=1).double()
    for got, want, S, n in ((dx, dp @ W.double(), dp.abs() @ W.double().abs(), 2 * F), (dW, dp.T @ x.double(), dp.abs().T @ x.double().abs(), N)):
        tol = 2 * U * n * S
        within(got, want, tol + (want.abs() + tol) * HALF[BF] + 2.0 ** -118)
    again = m.molora_gated_linear_backward(x, W, dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dW)


def wide_product(x, W):
    return sum(x[:, c:c + (1 << 14)].double() @ W[:, c:c + (1 << 14)].double().T for c in range(0, x.shape[1], 1 << 14))


def test_wide_inputs_do_not_drift(m):
    """The projections' sums run over d_in, in the forward pass (h has two of them as factors) and in dproj."""
    g, d = gen(72), 1 << 17
    x, W = (positive(g, 8192, d, by_row=True) / 256).to(BF), positive(g, 1024, d, by_row=True)
    h = m.molora_gated_linear(x, W, act="none")
    p = wide_product(x, W)
    off, most = drift(h, p[:, :512] * p[:, 512:])
    assert off <= most + 2.0 ** -15, (off, most)
    dh = positive(g, 2048, 512)
    _, _, dproj = m.molora_gated_linear_backward(x[:2048], W, dh, act="none", want_dx=False, want_dW=False)
    off, most = drift(dproj, torch.stack([p[:2048, 512:], p[:2048, :512]], dim=1) * dh.double()[:, None])
    assert off <= most, (off, most)


@pytest.mark.parametrize("N, d, F", [(9000, 8192, 264), (9000, 8200, 265), (9001, 20000, 250)])
def test_projections_of_long_sums(m, N, d, F):
    """d_in of one chain of K blocks, one more, several: g and u are within 2 u d S, S = sum |x w|, of their 64-bit sums, and
    SiLU's slope is 1.1 at most."""
    g = gen(d)
    x, W, dh = randn(g, N, d).to(BF), (randn(g, 2 * F, d) / math.sqrt(d)).to(BF), randn(g, N, F).to(BF)
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = m.molora_gated_linear(x, W, err_word=e)
    _, _, dproj = m.molora_gated_linear_backward(x, W, dh, want_dx=False, want_dW=False, err_word=e)
    assert e.item() == 0
    gate, up = wide_product(x, W).split(F, dim=1)
    eg, eu = (2 * U * d * wide_product(x.abs(), W.abs())).split(F, dim=1)
    p, dh = torch.sigmoid(gate), dh.double()
    a, s = gate * p, p + gate * p * (1 - p)
    want, tol = a * up, (1.1 * eg + 16 * U * gate.abs()) * (up.abs() + eu) + a.abs() * eu + 32 * U * (a * up).abs()
    within(h, want, tol + (want.abs() + tol) * HALF[BF])
    # (SiLU's second derivative is 1/2 at most; what rounds: the powers and factors, 256 u of each of two terms)
    want, tol = dh * up * s, dh.abs() * (up.abs() * (768 * U + 0.5 * eg) + 1.1 * eu)
    within(dproj[:, 0, :F], want, tol + (want.abs() + tol) * HALF[BF] + 2.0 ** -118)
    want, tol = dh * a, dh.abs() * (1.1 * eg + 256 * U * a.abs())
    within(dproj[:, 1, :F], want, tol + (want.abs() + tol) * HALF[BF] + 2.0 ** -118)
    assert torch.equal(m.molora_gated_linear(x, W), h)


# ---------------------------------------------------------------------------------------- quantiser
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, d", [(4096, 4096), (700, 1030), (16, 70001), (5000, 64)])
def test_quantised_values_are_the_quotients(m, dtype, N, d):
    """scale8 is the quotient of the largest magnitude and 448, and out8 x / scale8, each rounded to fp32 once and out8 then to
    e4m3, bit for bit (the expectation: IEEE divisions on the CPU), on values that are often halfway between two of e4m3."""
    g = gen(d)
    x = randn(g, N, d) * torch.exp2(torch.randint(-60, 60, (N, 1), generator=g, device="cuda").float())
    x[::3] = (x[::3].to(BF).float().view(torch.int32) & ~0xfffff).view(F32)  # few bits: more of them halfway
    x = x.to(dtype)
    x[:, 5::9], x[:, 3::11] = 0.0, -0.0
    out8, scale8 = m.molora_quantise_blocks(x)
    c = torch.nn.functional.pad(x.float().cpu(), (0, -d % 128)).view(N, -1, 128)
    scale = torch.div(c.abs().amax(2).clamp_min(2.0 ** -64), torch.full((1,), 448.0))
    want = (torch.div(c, scale[:, :, None]) + torch.where(c == 0, 0.0, -0.0)).clamp(-448, 448).view(N, -1)[:, :d].to(FP8)  # (-0: 0)
    assert torch.equal(scale8.cpu(), scale)
    assert torch.equal(out8.cpu().view(torch.uint8), want.view(torch.uint8))


def test_scales_of_every_largest_value(m):
    """Blocks of one value each: every finite bf16 magnitude, and fp32 ones of all sizes."""
    v = torch.arange(0x7f80, dtype=torch.int32).to(torch.int16).view(BF)
    g = torch.Generator().manual_seed(4)
    f = torch.randint(0, 0x7f800000, (1 << 18,), generator=g, dtype=torch.int32).view(F32)
    for x in (v, f):
        out8, scale8 = m.molora_quantise_blocks(x.view(-1, 1).cuda())
        scale = torch.div(x.float().clamp_min(2.0 ** -64), torch.full((1,), 448.0))
        assert torch.equal(scale8.cpu()[:, 0], scale)
        want = torch.div(x.float(), scale).clamp(-448, 448).to(FP8)
        assert torch.equal(out8.cpu()[:, 0].view(torch.uint8), want.view(torch.uint8))
