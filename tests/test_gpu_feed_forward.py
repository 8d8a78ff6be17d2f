"""The block-scaled product with its quantiser and the gated feed-forward block, forward and backward, against plain
64-bit implementations of their formulas.

Tolerances, derived from the arithmetic (u = 2^-24, half a step of fp32; half a step of bf16 is 2^-8 and of e4m3
2^-4 of the value, 2^-10 below its normal range):
  * quantiser: the scale is one division (u); the value is multiplied by a rounded reciprocal (u + u) and rounds to e4m3.
  * sums on the tensor cores: each of n additions loses at most a whole step (2 u) of a partial sum, itself at most
    S = sum |x w|: 2 u n S.  Blocks of 128 are scaled by a rounded product of two scales and added by one fma each:
    (2 u 128 + u (blocks + 4)) S, with S of the scaled operands.
  * epilogue: bias and activation (whose slope is at most 1.13) add 16 u of what they handle; outputs round once.
  * gated: with errors eg, eu of g and u, act(g) u is off by 1.13 eg (|u| + eu) + |act(g)| eu + 32 u |h|.
  * backward: act' is a sum of two terms that are 3 together at most, each within 256 u (an exponent of up to 126 and its
    factors within 2 u each); act'' is at most 1.2.  dg = dh u act'(g) is off by |dh| (|u| (768 u + 1.2 eg) + 1.13 eu),
    du = dh act(g) by |dh| (1.13 eg + 256 u |act(g)|); both round once.  dx and dW are sums of 2 d_ff and N products of
    dproj as stored.
Small integers, whose every partial sum is exact, have to come out bit for bit."""

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
    i = int(over.argmax()) if over.numel() else 0
    assert over.numel() == 0 or over.flatten()[i] <= 0, \
        f"element {i}: got {got.double().flatten()[i].item()}, want {want.flatten()[i].item()}, tolerance " \
        f"{torch.as_tensor(tol, device='cuda').broadcast_to(want.shape).flatten()[i].item()}"


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def guarded(shape, dtype, shift=0):
    """An output of this shape inside a buffer of a sentinel (shift: elements past a 16-byte boundary), and a check that
    nothing around it has been written."""
    n = math.prod(shape)
    buf = torch.full((n + 64 + shift,), 3.0, device="cuda").to(dtype)
    out = buf[shift:shift + n].view(shape)

    def untouched():
        assert (buf[shift + n:].float() == 3.0).all() and (buf[:shift].float() == 3.0).all()
    return out, untouched


def beside_nan(t):
    """t as the first part of a buffer whose rest is NaN: what is read past its end shows."""
    buf = torch.full((t.numel() + 4096,), math.nan, device="cuda").to(t.dtype)
    buf[:t.numel()] = t.flatten()
    return buf[:t.numel()].view(t.shape)


def blocks(n):
    return (n + 127) // 128


def spread(scale, rows, cols):
    if scale.shape[0] != rows:
        scale = scale.repeat_interleave(128, dim=0)[:rows]
    return scale.double().repeat_interleave(128, dim=1)[:, :cols]


def e4m3(g, rows, cols, row_blocks):
    """Random e4m3 values and positive scales of very different sizes."""
    v = (randn(g, rows, cols) * 100).clamp(-448, 448).to(FP8)
    return v, torch.exp2(2 * randn(g, row_blocks, blocks(cols)) - 6)


# ---------------------------------------------------------------------------------------- quantiser
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, d", [(1, 1), (1, 128), (3, 127), (2, 129), (5, 8), (16, 4096), (7, 4104), (33, 200), (1000, 1030),
                                  (5000, 512), (20000, 64), (3, 70001)])
def test_quantise(m, dtype, N, d):
    g = gen(N + d)
    x = (randn(g, N, d) * torch.exp(4 * randn(g, N, 1))).to(dtype)
    x[0, 0] = 0.0
    out, free = guarded((N, d), FP8)
    out8, scale8 = m.molora_quantise_blocks(beside_nan(x), out8=out)
    nb = blocks(d)
    amax = torch.nn.functional.pad(x.double().abs(), (0, nb * 128 - d)).view(N, nb, 128).amax(2)
    want = amax.clamp_min(2.0 ** -64) / 448
    within(scale8, want, want * 2 * U)
    q = x.double() / spread(want, N, d)
    within(out8.float(), q, q.abs() * (2.0 ** -4 + 8 * U) + 2.0 ** -10)
    free()


def test_quantise_special_values(m):
    x = torch.zeros(6, 300, device="cuda")
    x[1, 130] = math.inf
    x[2, 299] = math.nan
    x[3] = 2.0 ** -100
    x[4, :128] = 448.0
    x[4, 128:256] = -1e30
    x[5, 3], x[5, 4] = -math.inf, 7.0
    out8, s = m.molora_quantise_blocks(x)
    v = out8.float()
    low = 2.0 ** -64 / 448
    assert torch.equal(s[0], torch.full((3,), low, device="cuda")) and (v[0] == 0).all()
    assert s[1, 1] == math.inf and torch.isnan(v[1, 130]) and (v[1, 128:130] == 0).all() and s[1, 0].item() == pytest.approx(low)
    assert torch.isnan(s[2, 2]) and torch.isnan(v[2, 256:]).all() and (v[2, :256] == 0).all()
    assert (v[3] == 0).all()
    assert s[4, 0] == 1.0 and (v[4, :128] == 448).all() and (v[4, 128:256] == -448).all()
    assert s[5, 0] == math.inf and torch.isnan(v[5, 3]) and v[5, 4] == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantise_unaligned_rows(m, dtype):
    g = gen(5)
    x = randn(g, 40, 264).to(dtype)
    a, s = m.molora_quantise_blocks(x)
    buf = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")
    y = buf[1:].view(x.shape)
    y.copy_(x)
    out, free = guarded(x.shape, FP8, shift=3)
    b, t = m.molora_quantise_blocks(y, out8=out)
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(s, t)
    free()


# ---------------------------------------------------------------------------------------- block-scaled product
def blocks64(x, sx, W, sw, b, act, res):
    """The product and its tolerance before y's rounding."""
    a, w = x.double() * spread(sx, *x.shape), W.double() * spread(sw, *W.shape)
    v, S = a @ w.T, a.abs() @ w.abs().T
    tol = S * (256 * U + U * (blocks(x.shape[1]) + 4))
    if b is not None:
        v = v + b.double()
    y = ACTS[act](v)
    tol = 1.13 * tol + 16 * U * (v.abs() + y.abs())
    if res is not None:
        y = y + res.double()
        tol = tol + U * y.abs()
    return y, tol


@pytest.mark.parametrize("y_dtype", [BF, F32])
@pytest.mark.parametrize("d_in", [1024, 2304])
@pytest.mark.parametrize("d_out", [2047, 2056])
def test_linear_blocks_many_tiles_a_pair(m, y_dtype, d_in, d_out):
    """More tiles than pairs of CTAs, of one span of scales and of two, with a bias for each column: every call the same bits."""
    N, g = 3001, gen(d_in + d_out)
    x, sx = e4m3(g, N, d_in, N)
    W, sw = e4m3(g, d_out, d_in, blocks(d_out))
    b, res = 100 * randn(g, d_out), (100 * randn(g, N, d_out)).to(y_dtype)
    run = lambda: m.molora_linear_blocks(x, sx, W, sw, bias=beside_nan(b), act="silu", residual=res, out_dtype=y_dtype)  # noqa: E731
    y = run()
    want, tol = blocks64(x, sx, W, sw, b, "silu", res)
    within(y, want, tol + (want.abs() + tol) * HALF[y_dtype])
    assert all(torch.equal(run(), y) for _ in range(10))


@pytest.mark.parametrize("y_dtype", [BF, F32])
@pytest.mark.parametrize("N, d_in, d_out", [(1, 16, 1), (1, 4096, 512), (3, 128, 130), (16, 272, 64), (17, 2064, 257), (33, 512, 8),
                                            (64, 1024, 300), (100, 144, 1000), (129, 640, 384), (257, 256, 128), (300, 1040, 520),
                                            (512, 512, 2048), (1237, 2064, 1541), (2100, 384, 2304), (4096, 128, 1000), (5000, 48, 320)])
@pytest.mark.parametrize("act, bias, residual", [("none", False, False), ("silu", True, True), ("gelu_tanh", True, False)])
def test_linear_blocks(m, y_dtype, N, d_in, d_out, act, bias, residual):
    g = gen(N + d_in + d_out)
    x, sx = e4m3(g, N, d_in, N)
    W, sw = e4m3(g, d_out, d_in, blocks(d_out))
    b = 100 * randn(g, d_out) if bias else None
    res = (100 * randn(g, N, d_out)).to(y_dtype) if residual else None
    out, free = guarded((N, d_out), y_dtype)
    e = err_word()
    y = m.molora_linear_blocks(beside_nan(x), beside_nan(sx), beside_nan(W), beside_nan(sw), y=out, bias=b, act=act, residual=res, err_word=e)
    want, tol = blocks64(x, sx, W, sw, b, act, res)
    within(y, want, tol + (want.abs() + tol) * HALF[y_dtype])
    free()
    assert e.item() == 0
    again = m.molora_linear_blocks(x, sx, W, sw, bias=b, act=act, residual=res, out_dtype=y_dtype)
    assert torch.equal(y, again)


@pytest.mark.parametrize("N, d_in, d_out", [(1, 1024, 256), (40, 640, 264), (130, 4096, 136), (700, 384, 648), (3000, 272, 1160)])
def test_linear_blocks_exact_integers(m, N, d_in, d_out):
    g = gen(N)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()  # noqa: E731
    x, W = ints(N, d_in).to(FP8), ints(d_out, d_in).to(FP8)
    sx = torch.exp2(torch.randint(-2, 3, (N, blocks(d_in)), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-2, 3, (blocks(d_out), blocks(d_in)), generator=g, device="cuda").float())
    want, _ = blocks64(x, sx, W, sw, None, "none", None)
    y = m.molora_linear_blocks(x, sx, W, sw)
    assert torch.equal(y.double(), want)  # multiples of 1/16 below 2^20


@pytest.mark.parametrize("N", [5, 200, 1500])
@pytest.mark.parametrize("y_dtype", [BF, F32])
def test_linear_blocks_in_place_and_unaligned(m, N, y_dtype):
    """y as the residual itself, and y, residual, bias and scales off 16-byte boundaries: the same bits."""
    g = gen(N)
    d_in, d_out = 400, 640
    x, sx = e4m3(g, N, d_in, N)
    W, sw = e4m3(g, d_out, d_in, blocks(d_out))
    b, res = randn(g, d_out), (50 * randn(g, N, d_out)).to(y_dtype)
    want = m.molora_linear_blocks(x, sx, W, sw, bias=b, residual=res, out_dtype=y_dtype)
    y = res.clone()
    assert m.molora_linear_blocks(x, sx, W, sw, y=y, bias=b, residual=y) is y and torch.equal(y, want)

    def off(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v
    out, free = guarded((N, d_out), y_dtype, shift=1)
    m.molora_linear_blocks(x, off(sx), W, off(sw), y=out, bias=off(b), residual=off(res))
    assert torch.equal(out, want)
    free()


@pytest.mark.parametrize("N", [9, 150, 1100])
def test_linear_blocks_nan_stays_in_its_row(m, N):
    g = gen(N)
    d_in, d_out = 512, 520
    x, sx = e4m3(g, N, d_in, N)
    W, sw = e4m3(g, d_out, d_in, blocks(d_out))
    want = m.molora_linear_blocks(x, sx, W, sw)
    x2, sx2, W2, sw2 = x.clone(), sx.clone(), W.clone(), sw.clone()
    x2[3, 100] = math.nan
    sx2[5, 1] = math.inf
    W2[7, 9] = math.nan
    sw2[2, 0] = math.nan
    y = m.molora_linear_blocks(x2, sx2, W2, sw2)
    lost = torch.zeros(N, d_out, dtype=torch.bool, device="cuda")
    lost[3], lost[:, 7], lost[:, 256:384] = True, True, True
    assert torch.isnan(y[lost]).all()
    lost[5] = True
    assert not torch.isfinite(y[5]).any()
    assert torch.equal(y[~lost], want[~lost])


# ---------------------------------------------------------------------------------------- gated block, forward
def gated_inputs(g, dtype, N, d, F):
    if dtype == BF:
        return randn(g, N, d).to(BF), None, (randn(g, 2 * F, d) / math.sqrt(d)).to(BF), None
    x = (randn(g, N, d) * 40).clamp(-448, 448).to(FP8)
    W = (randn(g, 2 * F, d) * 40).clamp(-448, 448).to(FP8)
    sx = torch.exp2(0.5 * randn(g, N, blocks(d))) / 40
    sw = torch.exp2(0.5 * randn(g, 2 * blocks(F), blocks(d))) / (40 * math.sqrt(d))
    return x, sx, W, sw


def gated64(x, sx, W, sw, act):
    """h, g, u and the tolerances of h (before its rounding), g and u."""
    N, d = x.shape
    F = W.shape[0] // 2
    a, Wg, Wu = x.double(), W[:F].double(), W[F:].double()
    if sx is not None:
        a = a * spread(sx, N, d)
        Wg, Wu = Wg * spread(sw[:blocks(F)], F, d), Wu * spread(sw[blocks(F):], F, d)
        rate = 256 * U + U * (blocks(d) + 4)
    else:
        rate = 2 * U * d
    gate, up = a @ Wg.T, a @ Wu.T
    eg, eu = rate * (a.abs() @ Wg.abs().T), rate * (a.abs() @ Wu.abs().T)
    v = ACTS[act](gate)
    h = v * up
    # (activate handles the gate itself within 16 u of it)
    return h, gate, up, (1.13 * eg + 16 * U * (gate.abs() + v.abs())) * (up.abs() + eu) + v.abs() * eu + 32 * U * h.abs(), eg, eu


SIZES = [(1, 16, 1), (1, 2048, 640), (2, 128, 7), (16, 64, 33), (7, 1040, 64), (17, 272, 65), (33, 512, 200), (64, 2048, 1000),
         (100, 144, 130), (129, 640, 384), (257, 256, 128), (300, 1040, 777), (600, 512, 1000), (1237, 208, 1365), (2100, 256, 2304),
         (4096, 64, 520), (5000, 48, 96)]


@pytest.mark.parametrize("dtype", [BF, FP8])
@pytest.mark.parametrize("N, d, F", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_linear(m, dtype, N, d, F, act):
    g = gen(N + d + F)
    x, sx, W, sw = gated_inputs(g, dtype, N, d, F)
    want, _, _, tol, _, _ = gated64(x, sx, W, sw, act)
    e = err_word()
    out, free = guarded((N, F), BF)
    scales = {} if dtype == BF else dict(x_scale=beside_nan(sx), w_scale=beside_nan(sw))
    h = m.molora_gated_linear(beside_nan(x), beside_nan(W), h=out, act=act, err_word=e, **scales)
    assert h is out and e.item() == 0
    within(h, want, tol + (want.abs() + tol) * HALF[BF])
    free()
    assert torch.equal(m.molora_gated_linear(x, W, act=act, x_scale=sx, w_scale=sw), h)


@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, FP8])
@pytest.mark.parametrize("N", [3, 90, 900])
def test_gated_linear_activations(m, act, dtype, N):
    g = gen(N)
    x, sx, W, sw = gated_inputs(g, dtype, N, 256, 520)
    want, _, _, tol, _, _ = gated64(x, sx, W, sw, act)
    h = m.molora_gated_linear(x, W, act=act, x_scale=sx, w_scale=sw)
    within(h, want, tol + (want.abs() + tol) * HALF[BF])


@pytest.mark.parametrize("dtype", [BF, FP8])
@pytest.mark.parametrize("N, d, F", [(1, 512, 72), (20, 2048, 130), (200, 768, 264), (900, 400, 648), (2600, 256, 1096)])
def test_gated_linear_exact_integers(m, dtype, N, d, F):
    g = gen(N)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, W = ints(N, d), ints(2 * F, d)
    sx = sw = None
    if dtype == FP8:
        sx = torch.exp2(torch.randint(0, 2, (N, blocks(d)), generator=g, device="cuda").float())
        sw = torch.exp2(torch.randint(0, 2, (2 * blocks(F), blocks(d)), generator=g, device="cuda").float())
    want, gate, up, _, _, _ = gated64(x, sx, W, sw, "relu")
    h = m.molora_gated_linear(x, W, act="relu", x_scale=sx, w_scale=sw)
    assert gate.abs().max() < 2 ** 20
    # relu(g) u rounds to fp32, then to bf16
    assert torch.equal(h, (torch.relu(gate.float()) * up.float()).to(BF))


@pytest.mark.parametrize("dtype", [BF, FP8])
@pytest.mark.parametrize("N", [4, 150, 1100])
def test_gated_linear_unaligned_and_nan(m, dtype, N):
    g = gen(N)
    x, sx, W, sw = gated_inputs(g, dtype, N, 256, 264)
    kw = {} if dtype == BF else dict(x_scale=sx, w_scale=sw)
    want = m.molora_gated_linear(x, W, **kw)
    out, free = guarded((N, 264), BF, shift=1)
    m.molora_gated_linear(x, W, h=out, **kw)
    assert torch.equal(out, want)
    free()
    x2, W2 = x.clone(), W.clone()
    x2[2, 7] = math.nan
    W2[11, 3] = math.nan        # a gate's row
    W2[264 + 40, 250] = math.nan  # an up projection's
    h = m.molora_gated_linear(x2, W2, **kw)
    lost = torch.zeros_like(want, dtype=torch.bool)
    lost[2], lost[:, 11], lost[:, 40] = True, True, True
    assert torch.isnan(h[lost]).all() and torch.equal(h[~lost], want[~lost])


# ---------------------------------------------------------------------------------------- gated block, backward
def slope64(v, act):
    v = v.detach().clone().requires_grad_()
    ACTS[act](v).sum().backward()
    return v.grad


def check_backward(m, x, W, dh, act, **kw):
    N, d = x.shape
    F = W.shape[0] // 2
    e = err_word()
    _, g, u, _, eg, eu = gated64(x, None, W, None, act)
    dx, dW, dproj = m.molora_gated_linear_backward(x, W, dh, act=act, err_word=e, **kw)
    assert e.item() == 0
    dh, s, a, tiny = dh.double(), slope64(g, act), ACTS[act](g), 2.0 ** -118
    dg, du = dproj[:, 0, :F], dproj[:, 1, :F]
    if act == "relu":  # a gate within eg of 0 may fall on either side of it
        s, near = torch.where(g.abs() <= eg, torch.nan, s), g.abs() <= eg
        dg = torch.where(near, 0.0, dg.double())
        s = torch.where(near, 0.0, s)
    tol = dh.abs() * (u.abs() * (768 * U + 1.2 * eg) + 1.13 * eu)
    within(dg, dh * u * s, tol + ((dh * u * s).abs() + tol) * HALF[BF] + tiny)
    tol = dh.abs() * (1.13 * eg + 256 * U * a.abs())
    within(du, dh * a, tol + ((dh * a).abs() + tol) * HALF[BF] + tiny)
    dp = torch.cat([dproj[:, 0, :F], du], dim=1).double()
    if dx is not None:
        want, S = dp @ W.double(), dp.abs() @ W.double().abs()
        tol = 2 * U * 2 * F * S
        within(dx, want, tol + (want.abs() + tol) * HALF[BF] + tiny)
    if dW is not None:
        want, S = dp.T @ x.double(), dp.abs().T @ x.double().abs()
        tol = 2 * U * N * S
        within(dW, want, tol + (want.abs() + tol) * HALF[BF] + tiny)
    return dx, dW, dproj


@pytest.mark.parametrize("N, d, F", [(1, 8, 1), (3, 64, 7), (16, 128, 64), (64, 72, 65), (65, 264, 130), (129, 512, 200), (300, 1032, 777),
                                     (777, 136, 1365), (1024, 512, 512), (2500, 640, 384), (1500, 2048, 640)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_backward(m, N, d, F, act):
    g = gen(N + d + F)
    x, _, W, _ = gated_inputs(g, BF, N, d, F)
    dh = randn(g, N, F).to(BF)
    dx, free_x = guarded((N, d), BF)
    dW, free_w = guarded((2 * F, d), BF)
    dproj, free_p = guarded((N, 2, (F + 7) // 8 * 8), BF)
    out = check_backward(m, beside_nan(x), beside_nan(W), beside_nan(dh), act, dx=dx, dW=dW, dproj=dproj)
    free_x(), free_w(), free_p()
    # one of the two alone, and dh off 16-byte boundaries: the same bits
    a, none, _ = m.molora_gated_linear_backward(x, W, dh, act=act, want_dW=False)
    assert none is None and torch.equal(a, out[0])
    off = torch.empty(N * F + 1, dtype=BF, device="cuda")[1:].view(N, F)
    off.copy_(dh)
    none, b, dp = m.molora_gated_linear_backward(x, W, off, act=act, want_dx=False)
    assert none is None and torch.equal(b, out[1]) and torch.equal(dp[:, :, :F], out[2][:, :, :F])


@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
def test_gated_backward_activations(m, act):
    g = gen(3)
    x, _, W, _ = gated_inputs(g, BF, 200, 256, 520)
    check_backward(m, x, W, randn(g, 200, 520).to(BF), act)


@pytest.mark.parametrize("act", list(ACTS))
def test_slopes_over_the_whole_range(m, act):
    """dproj where the activation saturates, overflows or underflows: every finite bf16 gate, as one product with 1."""
    v = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(BF)
    v = v[torch.isfinite(v)]
    v = v[(v == 0) | (v.abs() >= 2.0 ** -120)]  # (fp32 powers flush what is smaller)
    F = v.numel()
    x = torch.zeros(1, 8, dtype=BF, device="cuda")
    x[0, 0] = 1
    W = torch.zeros(2 * F, 8, dtype=BF, device="cuda")
    W[:F, 0], W[F:, 0] = v, 1
    dh = torch.ones(1, F, dtype=BF, device="cuda")
    _, _, dproj = m.molora_gated_linear_backward(x, W, dh, act=act, want_dW=False)
    a, s = ACTS[act](v.double()), slope64(v.double(), act)
    if act == "gelu_tanh":  # (v^3 past fp64's square of it, 0 times infinity in the formula's gradient: saturated)
        s = torch.where(torch.isfinite(s), s, (v > 0).double())
    within(dproj[0, 0, :F], s, 3 * 256 * U + s.abs() * HALF[BF])
    # p within 256 u of itself, but flushed below 2^-126, where v p is below 2^-119
    within(dproj[0, 1, :F], a, a.abs() * (HALF[BF] + 256 * U) + 2.0 ** -118)


@pytest.mark.parametrize("N, d, F", [(5, 64, 24), (200, 264, 136), (900, 136, 1000), (2000, 512, 256)])
def test_gated_backward_exact_integers(m, N, d, F):
    """Sparse small integers, so that the projections, dproj (below 256) and the sums are exact."""
    g = gen(N)

    def ints(*s):
        return (torch.randint(-1, 2, s, generator=g, device="cuda") * (torch.rand(s, generator=g, device="cuda") < 0.1)).to(BF)
    x, W, dh = ints(N, d), ints(2 * F, d), torch.randint(-1, 2, (N, F), generator=g, device="cuda").to(BF)
    dx, dW, dproj = m.molora_gated_linear_backward(x, W, dh, act="relu")
    gate, up = (x.double() @ W.double().T).split(F, dim=1)
    dp = torch.cat([dh.double() * up * (gate > 0), dh.double() * torch.relu(gate)], dim=1)
    assert dp.abs().max() <= 256
    assert torch.equal(torch.cat([dproj[:, 0, :F], dproj[:, 1, :F]], dim=1).double(), dp)
    assert torch.equal(dx, (dp @ W.double()).float().to(BF))
    assert torch.equal(dW, (dp.T @ x.double()).float().to(BF))


def test_gated_gradient_against_differences(m):
    """<dx, v> + <dW, V> against (L(x + e v, W + e V) - L(x - e v, W - e V)) / 2 e of L = sum h dh in 64 bits.  The central
    difference is off by e^2 / 6 of a third derivative, 1e-9 here, and by 2^-53 of L / e.  dproj, dx and dW round to bf16, by
    2^-8 of themselves at most and in either direction: six deviations of what these roundings sum to."""
    g = gen(8)
    N, d, F = 48, 64, 40
    x, _, W, _ = gated_inputs(g, BF, N, d, F)
    dh = randn(g, N, F).to(BF)
    for act in ("silu", "gelu", "gelu_tanh"):
        dx, dW, dproj = m.molora_gated_linear_backward(x, W, dh, act=act)
        v, V = randn(g, N, d).double(), randn(g, 2 * F, d).double() / math.sqrt(d)

        def loss(e):
            a, w = x.double() + e * v, W.double() + e * V
            return (ACTS[act](a @ w[:F].T) * (a @ w[F:].T) * dh.double()).sum()
        e = 1e-5
        want = (loss(e) - loss(-e)) / (2 * e)
        got = (dx.double() * v).sum() + (dW.double() * V).sum()
        dp = torch.cat([dproj[:, 0, :F], dproj[:, 1, :F]], dim=1).double()
        rounded = [dp * (v @ W.double().T + x.double() @ V.T), dx.double() * v, dW.double() * V]
        deviation = HALF[BF] * sum(r.pow(2).sum() for r in rounded).sqrt()
        assert abs(got - want) <= 6 * deviation + 1e-6


def test_gated_backward_of_nothing(m):
    W = torch.randn(48, 16, device="cuda").to(BF)
    x, dh = torch.empty(0, 16, dtype=BF, device="cuda"), torch.empty(0, 24, dtype=BF, device="cuda")
    assert m.molora_gated_linear(x, W).shape == (0, 24)
    dW = torch.ones_like(W)
    dx, dW, dproj = m.molora_gated_linear_backward(x, W, dh, dW=dW)
    assert dx.shape == (0, 16) and dproj.shape == (0, 2, 24) and (dW == 0).all()
    x8 = torch.empty(0, 16, dtype=FP8, device="cuda")
    assert m.molora_linear_blocks(x8, torch.empty(0, 1, device="cuda"), W.to(FP8), torch.ones(1, 1, device="cuda")).shape == (0, 48)
    assert m.molora_quantise_blocks(x)[0].shape == (0, 16)


# ---------------------------------------------------------------------------------------- together
def test_feed_forward_half_in_bf16_and_in_blocks(m):
    """norm -> gated block -> product down with the residual, in bf16 and in block-scaled e4m3 of the same weights, over
    a prefill and one token of it, captured and replayed with other inputs."""
    g = gen(21)
    N, d, F = 384, 512, 1000
    Fp = 1008  # (the way down's d_in: a multiple of 16, the gated block's columns padded with rows of zeros)
    nw = (1 + 0.1 * randn(g, d)).to(BF)
    W = randn(g, 2 * Fp, d) / math.sqrt(d)
    W[F:Fp], W[Fp + F:] = 0, 0
    Wd = randn(g, d, Fp) / math.sqrt(F)

    def weights8(w):
        r, c = w.shape
        amax = torch.nn.functional.pad(w.abs(), (0, blocks(c) * 128 - c, 0, blocks(r) * 128 - r)).view(blocks(r), 128, blocks(c), 128)
        s = amax.amax(3).amax(1).clamp_min(2.0 ** -64) / 448
        return (w / spread(s, r, c).float()).to(FP8), s
    (g8, gs), (u8, us), (d8, ds) = weights8(W[:Fp]), weights8(W[Fp:]), weights8(Wd)
    W8, ws = torch.cat([g8, u8]), torch.cat([gs, us])

    def half16(x):
        _, n, _, _ = m.molora_rmsnorm(x, nw)
        h = m.molora_gated_linear(n, W.to(BF))
        return m.molora_linear(h, Wd.to(BF), residual=x, out_dtype=BF)

    def half8(x):
        _, n, _, _ = m.molora_rmsnorm(x, nw)
        n8, ns = m.molora_quantise_blocks(n)
        h = m.molora_gated_linear(n8, W8, x_scale=ns, w_scale=ws)
        h8, hs = m.molora_quantise_blocks(h)
        return m.molora_linear_blocks(h8, hs, d8, ds, residual=x, out_dtype=BF)

    def half64(x):
        s = x.double()
        n = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * nw.double()
        return s + (ACTS["silu"](n @ W[:Fp].double().T) * (n @ W[Fp:].double().T)) @ Wd.double().T

    for rows in (N, 1):
        x = randn(g, rows, d).to(BF)
        want = half64(x)
        update = (want - x.double()).pow(2).mean().sqrt()
        # rms: bf16 rounds n, W, h, Wd and y (2^-9 each, at most 2^-8); e4m3 n, W, h and Wd by 2^-4 at most, 2^-5 or so on average
        assert (half16(x).double() - want).pow(2).mean().sqrt() <= 6 * 2.0 ** -8 * (update + 1)
        assert (half8(x).double() - want).pow(2).mean().sqrt() <= 4 * 2.0 ** -4 * update
        for half in (half16, half8):
            buf = x.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                half(buf)
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = half(buf)
            for _ in range(2):
                buf.copy_(randn(g, rows, d).to(BF))
                graph.replay()
                assert torch.equal(y, half(buf))


def test_adapters_train_through_a_frozen_block(m):
    """An adapter on the way down of a frozen block: the block's dx, with no gradient of its weights, equals the one that the
    whole backward pass gives, on a stream of the caller's."""
    g = gen(30)
    N, d, F = 200, 256, 320
    x, _, W, _ = gated_inputs(g, BF, N, d, F)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = m.molora_gated_linear(x, W, stream=side)
    dh = randn(g, N, F).to(BF)
    side.wait_stream(torch.cuda.current_stream())
    dx, dW, dproj = m.molora_gated_linear_backward(x, W, dh, want_dW=False, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for t in (h, dx, dproj):
        t.record_stream(torch.cuda.current_stream())
    want, _, _ = m.molora_gated_linear_backward(x, W, dh)
    assert dW is None and torch.equal(dx, want)


@pytest.mark.parametrize("kind", ["quantise", "blocks", "gated", "gated_fp8", "backward"])
def test_offsets_past_32_bits(m, kind):
    """Outputs (and, of the quantiser, inputs) of more than 2^31 elements: the first, the middle and the last rows."""
    g = gen(50)
    rows = lambda N: torch.tensor([0, 1, N // 2 - 1, N // 2, N // 2 + 1, N - 2, N - 1], device="cuda")  # noqa: E731
    if kind == "quantise":
        N, d = 530000, 4096
        x = torch.zeros(N, d, dtype=BF, device="cuda")
        at = rows(N)
        x[at] = randn(g, 7, d).to(BF)
        out8, scale8 = m.molora_quantise_blocks(x)
        a, b = m.molora_quantise_blocks(x[at].contiguous())
        assert torch.equal(out8[at].view(torch.uint8), a.view(torch.uint8)) and torch.equal(scale8[at], b)
        return
    if kind == "backward":
        N, d, F = 280000, 64, 4096
        x, _, W, _ = gated_inputs(g, BF, N, d, F)
        dh = torch.zeros(N, F, dtype=BF, device="cuda")
        at = rows(N)
        dh[at] = randn(g, 7, F).to(BF)
        dx, dW, dproj = m.molora_gated_linear_backward(x, W, dh)
        a, b, c = m.molora_gated_linear_backward(x[at].contiguous(), W, dh[at].contiguous())
        assert torch.equal(dproj[at], c) and (dx[2:1000] == 0).all()
        # (few and many tokens' dx take other kernels: fp32 sums of 2 F terms in another order, and a rounding of either)
        dp = torch.cat([c[:, 0], c[:, 1]], dim=1).double()
        want, tol = dp @ W.double(), 2 * U * 2 * F * (dp.abs() @ W.double().abs())
        for got in (dx[at], a):
            within(got, want, tol + (want.abs() + tol) * HALF[BF] + 2.0 ** -118)
        within(dW, b.double(), 2 * (b.double().abs() * HALF[BF]) + 2.0 ** -20)  # (the same 7 terms, in two orders of additions)
        return
    N, d, F = 530000, 128, 4096
    if kind == "blocks":
        x, sx = e4m3(g, N, d, N)
        W, sw = e4m3(g, F, d, blocks(F))
        run = lambda i: m.molora_linear_blocks(x[i].contiguous(), sx[i].contiguous(), W, sw, out_dtype=BF)  # noqa: E731
    else:
        x, sx, W, sw = gated_inputs(g, FP8 if kind == "gated_fp8" else BF, N, d, F)
        run = lambda i: m.molora_gated_linear(x[i].contiguous(), W, x_scale=None if sx is None else sx[i].contiguous(), w_scale=sw)  # noqa: E731
    y = run(slice(None))
    few = run(rows(N))
    # (few and many tokens take other kernels: sums in another order, and a rounding of either)
    within(y[rows(N)], few.double(), few.double().abs() * 2 * HALF[BF] + 2.0 ** -10 * few.double().abs().mean())


def test_two_streams_and_two_graphs_at_once(m):
    """Calls on two streams at once, and two captured graphs of them replayed in turn, keep to their own buffers."""
    g = gen(60)
    jobs = []
    for N in (2000, 1100):
        x, sx = e4m3(g, N, 512, N)
        W, sw = e4m3(g, 1024, 512, 8)
        b, _, V, _ = gated_inputs(g, BF, N, 256, 768)
        dh = randn(g, N, 768).to(BF)

        def run(x=x, sx=sx, W=W, sw=sw, b=b, V=V, dh=dh):
            return [m.molora_linear_blocks(x, sx, W, sw), m.molora_gated_linear(b, V), *m.molora_gated_linear_backward(b, V, dh)]
        jobs.append(run)
    want = [run() for run in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, run in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, v in zip(want, got) for a, b in zip(w, v))
    graphs = []
    for run in jobs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out))
    for _ in range(2):
        for graph, out in graphs:
            for t in out:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, (_, v) in zip(want, graphs) for a, b in zip(w, v))
