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
