"""A wait whose time runs out sets DEV_WAIT_TIMEOUT and leaves no wrong number behind: the library is linked once
more with the waits of one warp of one CTA, after they completed, reported as run out (lost_waits.cu)."""

import concurrent.futures
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
OLD = 7.0  # what y holds before the call


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    """(the binding, its library, the library with waits that can be lost)"""
    from token_adapter_routing_gb300 import build
    import token_adapter_routing_gb300 as m
    build.build()
    lib = m.load_library()
    out = tmp_path_factory.mktemp("lost_waits")
    here = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lost_waits.cu")

    def compile_one(name):
        obj = str(out / (name + ".o"))
        subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, f'-DMOLORA_SOURCE="{name}.cu"',
                        f"-DMOLORA_SET=lost_in_{name}", "-c", here, "-o", obj], check=True)
        return obj
    names = ("linear", "lora_update")
    with concurrent.futures.ThreadPoolExecutor() as ex:
        objs = list(ex.map(compile_one, names))
    objs += [os.path.join(build.BUILD, os.path.basename(s)[:-3] + ".o") for s in build.sources()
             if os.path.basename(s)[:-3] not in names]
    path = str(out / "libmolora_lost.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", path, *objs], check=True)
    lost = ctypes.CDLL(path)
    for name in ("molora_linear", "molora_norm_linear_lora_apply"):
        getattr(lost, name).argtypes = getattr(lib, name).argtypes
    return m, lib, lost


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def linear(lib, x, W, sx, sw, y, e):
    code = {F32: 0, BF: 1, FP8: 2}[x.dtype]
    p = [None if t is None else t.data_ptr() for t in (x, sx, W, sw, y, e)]
    status = lib.molora_linear(p[0], code, p[1], x.shape[0], x.shape[1], p[2], p[3], W.shape[0], None, 0, None, p[4],
                               1 if y.dtype == BF else 0, p[5], torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()


def call_with_lost(libs, which, cta, warp, run):
    _, _, lost = libs
    pick = getattr(lost, f"lost_in_{which}")
    assert pick(cta, warp) == 0
    try:
        run(lost)
    finally:
        torch.cuda.synchronize()
        assert pick(-1, -1) == 0


# the split kernels (d_in over clusters of 4 and 8 CTAs, and over one): CTAs of tile 0, and every kind of warp
@pytest.mark.parametrize("dtype, N, d_in, d_out", [
    (BF, 16, 4096, 4096), (FP8, 16, 4096, 4096), (BF, 16, 2048, 256), (BF, 100, 2048, 256), (BF, 16, 128, 512),
    (FP8, 16, 256, 512), (F32, 16, 1024, 512), (F32, 16, 64, 512), (BF, 16, 1030, 512), (F32, 100, 1030, 512),
    (FP8, 16, 1030, 512)])
@pytest.mark.parametrize("cta, warp", [(0, 0), (0, 3), (1, 0), (1, 7), (0, -2), (1, -2)])
def test_split_product_loses_to_nan(libs, dtype, N, d_in, d_out, cta, warp):
    m, lib, _ = libs
    g = gen(d_in + N)
    x, W, sx, sw = randn(g, N, d_in), randn(g, d_out, d_in), None, None
    if dtype == FP8:
        sx, sw = torch.ones(N, device="cuda"), torch.ones(d_out, device="cuda")
    x, W = x.to(dtype), W.to(dtype)
    rows16 = d_in * x.element_size() % 16 == 0
    issuer = warp == -2
    if issuer:  # the warp that issues the MMAs
        warp = 9 if rows16 and dtype != F32 else 15
    if cta == 1 and d_in * (1 if dtype == FP8 and rows16 else 2) <= 256:
        pytest.skip("one CTA a tile: CTA 1 has a tile of its own")
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = torch.full((N, d_out), OLD, device="cuda")
    linear(lib, x, W, sx, sw, want, e)
    assert e.item() == 0
    y = torch.full((N, d_out), OLD, device="cuda")
    call_with_lost(libs, "linear", cta, warp, lambda lost: linear(lost, x, W, sx, sw, y, e))
    assert e.item() == m.DEV_WAIT_TIMEOUT
    # a tile is 16 tokens at least, of which warps 0 and 3 have outputs 0 .. 31 and 96 .. 127
    if dtype != F32 and (warp in (0, 3) or issuer):
        assert torch.isnan(y[:16, slice(128) if issuer else slice(32 * warp, 32 * warp + 32)]).all()
    same = y == want
    if dtype == F32:  # (whose NaN may be summed again, in another order; a lost share is off by a hundred times this)
        same |= (y - want).abs() <= 2.0 ** -23 * (d_in + 16) * (x.abs() @ W.abs().T)
    assert (same | torch.isnan(y)).all()
    assert torch.equal(y[:, 128:], want[:, 128:])
    # and nothing stays behind
    e.zero_()
    linear(libs[2], x, W, sx, sw, y, e)
    assert e.item() == 0 and torch.equal(y, want)


@pytest.mark.parametrize("y_dtype", [BF, F32])
@pytest.mark.parametrize("cta, warp", [(0, 0), (1, 5)])
def test_pair_product_writes_nothing_wrong(libs, y_dtype, cta, warp):
    m, lib, _ = libs
    g = gen(3)
    x, W = randn(g, 2048, 512).to(BF), randn(g, 1024, 512).to(BF)
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, y = (torch.full((2048, 1024), OLD, dtype=y_dtype, device="cuda") for _ in range(2))
    linear(lib, x, W, None, None, want, e)
    call_with_lost(libs, "linear", cta, warp, lambda lost: linear(lost, x, W, None, None, y, e))
    assert e.item() == m.DEV_WAIT_TIMEOUT
    assert ((y == want) | (y == OLD)).all()
    assert (y == OLD).any()


@pytest.mark.parametrize("K, r", [(4, 16), (7, 64)])
@pytest.mark.parametrize("cta, warp", [(0, 0), (1, 0), (1, 9), (0, 9), (1, 8)])
def test_update_that_was_lost_is_nan(libs, K, r, cta, warp):
    """The tokens whose update a shrink's run-out wait lost are NaN, whatever the workspace held; the others are right."""
    m, lib, _ = libs
    g = gen(K)
    N, d = 300, 512
    x, nw = randn(g, N, d).to(BF), torch.ones(d, dtype=BF, device="cuda")
    W = (randn(g, d, d) / d ** 0.5).to(BF)
    A, B = (randn(g, K, d, r) / d ** 0.5).to(BF), randn(g, K, r, d).to(BF)
    ids = (torch.arange(N, device="cuda") % K).to(torch.int32)
    w = torch.rand(N, generator=g, device="cuda")
    ws = torch.zeros(2 * ((N * K * r * 2 + 255) // 256 * 256), dtype=torch.uint8, device="cuda")

    def run(lib):
        h, y = torch.empty_like(x), torch.full((N, d), OLD, device="cuda")
        e = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = ctypes.c_size_t(ws.numel())
        p = [t.data_ptr() for t in (x, nw, h, W, A, B, ids, w, y, ws, e)]
        status = lib.molora_norm_linear_lora_apply(
            p[0], 1, N, d, None, None, p[1], 1e-6, p[2], None, None, p[3], 1, None, d, None, p[4], p[5], K, r, p[6], p[7], 1,
            None, None, None, 2.0, p[8], 0, p[9], ctypes.byref(size), p[10], torch.cuda.current_stream().cuda_stream)
        assert status == 0
        torch.cuda.synchronize()
        return y, e.item()
    want, e = run(lib)
    assert e == 0
    for stale in (0, 63):  # of bf16, 0 and 0.747
        ws.fill_(stale)
        out = []
        call_with_lost(libs, "lora_update", cta, warp, lambda lost: out.append(run(lost)))
        y, e = out[0]
        assert e == m.DEV_WAIT_TIMEOUT
        assert ((y == want) | torch.isnan(y)).all()
        assert torch.equal(y[128:], want[128:])  # tile 0 is 128 tokens; warp 0 has its first 32
        if warp in (0, 9):
            assert torch.isnan(y[:32 if warp == 0 else 128]).all()
