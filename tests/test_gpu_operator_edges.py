"""What the norm and the base product do with NaN, infinities, borders of rounding and long sums, beyond
test_gpu_operators.py."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


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


def off_by_one(t):
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


# rows in whole chunks (with and without the row ahead), off the 16-byte grid, read element by element, and long
NORMS = [(BF, 8, 192), (BF, 2500, 512), (F32, 8, 192), (BF, 37, 2049), (F32, 1237, 2049), (BF, 2, 70000), (F32, 3, 40000)]


@pytest.mark.parametrize("unaligned", [False, True])
@pytest.mark.parametrize("dtype, N, d", NORMS)
def test_norm_weight_nan_and_infinity(m, dtype, N, d, unaligned):
    """max |n| of a row with a NaN is NaN, and so is its scale; with an infinity it is infinite, and n / scale8 is 0
    at the finite elements and NaN at the infinite one."""
    g = gen(N + d)
    x = randn(g, N, d).sign().to(dtype) * (1 + torch.rand(N, d, generator=g, device="cuda")).to(dtype)  # nothing is 0
    x = off_by_one(x) if unaligned else x
    for at in (0, d // 2 + 1, d - 1):
        w = torch.ones(d, dtype=dtype, device="cuda")
        w[at] = math.nan
        out, out8 = torch.empty(N, d, dtype=dtype, device="cuda"), torch.empty(N, d, dtype=FP8, device="cuda")
        scale8 = torch.empty(N, device="cuda")
        m.molora_rmsnorm(x, w, out=out, out8=out8, scale8=scale8)
        odd = torch.isnan(out)
        assert odd[:, at].all() and odd.sum().item() == N
        assert torch.isnan(scale8).all() and torch.isnan(out8.float()).all()
        w[at] = -math.inf
        m.molora_rmsnorm(x, w, out=out, out8=out8, scale8=scale8)
        assert torch.equal(out[:, at].float(), -x[:, at].sign().float() * math.inf)
        assert torch.isinf(out).sum().item() == N and (scale8 == math.inf).all()
        o8 = out8.float()
        assert torch.isnan(o8[:, at]).all() and torch.isnan(o8).sum().item() == N
        assert (o8.nan_to_num(0.0) == 0).all()


@pytest.mark.parametrize("unaligned", [False, True])
@pytest.mark.parametrize("dtype, N, d", NORMS)
def test_norm_infinite_rows(m, dtype, N, d, unaligned):
    """An infinity makes the row's root infinite: NaN at the infinity itself, 0 at the finite elements, and a NaN
    scale, with which the whole row in 8 bits is NaN.  The other rows are what they are without it."""
    g = gen(N * 3 + d)
    x, w = randn(g, N, d).to(dtype), (1 + 0.1 * randn(g, d)).to(dtype)
    x = off_by_one(x) if unaligned else x

    def call():
        out8, scale8 = torch.empty(N, d, dtype=FP8, device="cuda"), torch.empty(N, device="cuda")
        out = m.molora_rmsnorm(x, w, out=torch.empty(N, d, dtype=dtype, device="cuda"), out8=out8, scale8=scale8)[1]
        return out, out8.float(), scale8
    plain = call()
    x[1, 7] = -math.inf
    out, out8, scale8 = call()
    assert torch.isnan(out[1, 7]) and torch.isnan(out).sum().item() == 1
    assert (out[1, :7] == 0).all() and (out[1, 8:] == 0).all()
    assert torch.isnan(scale8[1]) and torch.isnan(out8[1]).all()
    rest = [0] + list(range(2, N))
    for a, b in zip((out, out8, scale8), plain):
        assert torch.equal(a[rest], b[rest])


@pytest.mark.parametrize("N, d", [(4096, 2048), (3000, 2049), (40, 40000)])
def test_norm_out8_is_the_product_with_the_reciprocal(m, N, d):
    """out8 is e4m3(n * (1 / scale8)) of the fp32 n and scale8 that the call returns, to the bit."""
    g = gen(N)
    x, w = randn(g, N, d), 1 + 0.1 * randn(g, d)
    out8, scale8 = torch.empty(N, d, dtype=FP8, device="cuda"), torch.empty(N, device="cuda")
    out = m.molora_rmsnorm(x, w, out=torch.empty_like(x), out8=out8, scale8=scale8)[1]
    q = out.cpu() * (1.0 / scale8.cpu())[:, None]
    want = q.clamp(-448, 448).to(FP8)
    assert torch.equal(out8.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("N, d_in, d_out", [(5, 255, 33), (140, 256, 64), (64, 1024, 300), (1100, 512, 1032), (150, 1023, 70)])
def test_infinities_leave_the_neighbours_bits(m, N, d_in, d_out):
    """fp32: an infinity or NaN in one token, or one output's weights, changes no bit of the others."""
    g = gen(N + d_in)
    x, W = randn(g, N, d_in), randn(g, d_out, d_in) / math.sqrt(d_in)
    plain = m.molora_linear(x, W)
    bad = x.clone()
    bad[2, 4], bad[4, d_in - 1] = math.inf, math.nan
    bad.view(torch.int32)[1, 3] = 0x7f800001  # a NaN of low bits only
    y = m.molora_linear(bad, W)
    rest = [0, 3] + list(range(5, N))
    assert torch.equal(y[rest], plain[rest])
    assert torch.isnan(y[1]).all() and torch.isnan(y[4]).all()
    assert torch.equal(y[2], torch.where(W[:, 4] > 0, math.inf, -math.inf))
    V = W.clone()
    V[5, 7] = -math.inf
    y = m.molora_linear(x, V)
    cols = [i for i in range(d_out) if i != 5]
    assert torch.equal(y[:, cols], plain[:, cols])
    assert torch.equal(y[:, 5], torch.where(x[:, 7] > 0, -math.inf, math.inf))


@pytest.mark.parametrize("dtype, N, d_in, d_out", [
    (BF, 4096, 4096, 2048), (BF, 16, 4096, 10240), (F32, 1000, 4096, 4096), (BF, 1000, 4095, 4096), (F32, 1000, 4095, 4096),
    # d_in over several CTAs, and the CUDA cores
    (BF, 16, 4096, 4096), (BF, 300, 4096, 512), (F32, 64, 4096, 1024), (F32, 2, 4096, 1024)])
def test_long_sums_do_not_drift(m, dtype, N, d_in, d_out):
    """fp32 y of positive products, whose partial sums only grow.  A tensor core cuts what an addition loses, half a
    step (2^-24 of the sum or less) on the mean.  Sums of 32 MMAs that registers add lose 2^-24 sum_j j / 32 =
    1.0e-6 at most, and fp32's further products, 2^-7 of the first, 640 in a chain, 3e-7; one chain of 256 would
    lose 2^-25 sum_j j / 256 = 3.8e-6 at least."""
    g = gen(d_in)
    x = (0.5 + 0.5 * torch.rand(N, d_in, generator=g, device="cuda")).to(dtype)
    W = (0.5 + 0.5 * torch.rand(d_out, d_in, generator=g, device="cuda")).to(dtype)
    y = m.molora_linear(x, W).double()
    want = x.double() @ W.double().T
    drift = ((y - want) / want).mean().abs().item()
    assert drift <= 1.5e-6, drift


@pytest.mark.parametrize("N", [16, 300])
def test_an_empty_workspace_is_none(m, N):
    """A buffer of the 0 bytes that a size query may give: the calls run, as they do without one."""
    g = gen(N)
    d, K, r = 256, 4, 16
    x, nw = randn(g, N, d).to(BF), torch.ones(d, dtype=BF, device="cuda")
    W, A, B = randn(g, d, d).to(BF), randn(g, K, d, r).to(BF), randn(g, K, r, d).to(BF)
    ids = (torch.arange(N, device="cuda") % K).to(torch.int32)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    y, want = torch.ones(N, d, device="cuda"), torch.ones(N, d, device="cuda")
    m.molora_lora_apply(x, A, B, ids, want, 2.0, path="scalar")
    m.molora_lora_apply(x, A, B, ids, y, 2.0, path="scalar", ws=none)
    assert torch.equal(y, want) and not (y == 1).all()
    y.fill_(7.0)
    _, _, h, _, _ = m.molora_norm_linear_lora_apply(x, nw, 1e-6, W, A, B, ids, y, 2.0, ws=none)
    want = h.double() @ W.double().T
    for a in range(K):
        want += 2.0 * (ids == a).double()[:, None] * ((h.double() @ A[a].double()) @ B[a].double())
    assert (y.double() - want).abs().max() <= 2e-4 * want.pow(2).mean().sqrt()  # the apply's own bar
