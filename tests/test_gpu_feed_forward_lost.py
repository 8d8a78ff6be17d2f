"""A wait of the feed-forward kernels whose time runs out sets DEV_WAIT_TIMEOUT and leaves no wrong number behind: the
library is linked once more with the waits of one warp of one CTA, after they completed, reported as run out
(lost_waits.cu).  Few tokens: what was lost is NaN.  Many: what was lost stays as it was.  The backward pass: what was lost
of dproj is NaN, and so is what its products make of it."""

import concurrent.futures
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
OLD = 7.0  # what an output holds before the call
CALLS = ("molora_linear_blocks", "molora_gated_linear", "molora_gated_linear_backward")


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
    names = ("feed_forward", "blocks_tc", "gated_grad")
    with concurrent.futures.ThreadPoolExecutor() as ex:
        objs = list(ex.map(compile_one, names))
    objs += [os.path.join(build.BUILD, os.path.basename(s)[:-3] + ".o") for s in build.sources()
             if os.path.basename(s)[:-3] not in names]
    path = str(out / "libmolora_lost.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", path, *objs], check=True)
    lost = ctypes.CDLL(path)
    for name in CALLS:
        getattr(lost, name).argtypes = getattr(lib, name).argtypes
    return m, lib, lost


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def old(*shape, dtype=BF):
    return torch.full(shape, OLD, dtype=dtype, device="cuda")


def p(t):
    return None if t is None else t.data_ptr()


def call(fn, *args):
    assert fn(*args, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()


def with_lost(libs, which, cta, warp, run):
    """run(the library that loses waits), and what stays behind: nothing."""
    pick = getattr(libs[2], f"lost_in_{which}")
    assert pick(cta, warp) == 0
    try:
        run(libs[2])
    finally:
        torch.cuda.synchronize()
        assert pick(-1, -1) == 0


def blocks(lib, x, sx, W, sw, y, e):
    call(lib.molora_linear_blocks, p(x), p(sx), x.shape[0], x.shape[1], p(W), p(sw), W.shape[0], None, 0, None, p(y),
         1 if y.dtype == BF else 0, p(e))


def gated(lib, x, sx, W, sw, h, e):
    call(lib.molora_gated_linear, p(x), 2 if x.dtype == FP8 else 1, p(sx), x.shape[0], x.shape[1], p(W), p(sw), W.shape[0] // 2, 2, p(h), p(e))


def inputs(g, dtype, N, d, rows, row_blocks):
    x, W = randn(g, N, d).to(dtype), randn(g, rows, d).to(dtype)
    if dtype == BF:
        return x, None, W, None
    nb = (d + 127) // 128
    return x, 0.5 + torch.rand(N, nb, generator=g, device="cuda"), W, 0.5 + torch.rand(row_blocks, nb, generator=g, device="cuda")


@pytest.mark.parametrize("kind, dtype, N, d, F", [("blocks", FP8, 16, 2048, 512), ("blocks", FP8, 16, 128, 256), ("gated", FP8, 16, 2048, 512),
                                                  ("gated", BF, 16, 2048, 512), ("gated", BF, 100, 1024, 256)])
@pytest.mark.parametrize("cta, warp", [(0, 0), (0, 3), (1, 7), (0, 9), (1, 9)])
def test_few_tokens_lose_to_nan(libs, kind, dtype, N, d, F, cta, warp):
    m, lib, lost = libs
    g = gen(N + d)
    rb = (F + 127) // 128
    x, sx, W, sw = inputs(g, dtype, N, d, F if kind == "blocks" else 2 * F, rb if kind == "blocks" else 2 * rb)
    fn, e = (blocks if kind == "blocks" else gated), torch.zeros(1, dtype=torch.int32, device="cuda")
    want, y = old(N, F), old(N, F)
    fn(lib, x, sx, W, sw, want, e)
    assert e.item() == 0
    with_lost(libs, "feed_forward", cta, warp, lambda lib: fn(lib, x, sx, W, sw, y, e))
    assert e.item() == m.DEV_WAIT_TIMEOUT
    assert ((y == want) | torch.isnan(y)).all() and torch.isnan(y).any()
    e.zero_()
    fn(lost, x, sx, W, sw, y, e)
    assert e.item() == 0 and torch.equal(y, want)


@pytest.mark.parametrize("kind, dtype", [("blocks", FP8), ("gated", FP8), ("gated", BF)])
@pytest.mark.parametrize("cta, warp", [(0, 0), (1, 5), (0, 9)])
def test_many_tokens_write_nothing_wrong(libs, kind, dtype, cta, warp):
    m, lib, lost = libs
    g = gen(3)
    N, d, F = 2048, 1024, 2048
    x, sx, W, sw = inputs(g, dtype, N, d, F if kind == "blocks" else 2 * F, 16 if kind == "blocks" else 32)
    fn, e = (blocks if kind == "blocks" else gated), torch.zeros(1, dtype=torch.int32, device="cuda")
    want, y = old(N, F), old(N, F)
    fn(lib, x, sx, W, sw, want, e)
    with_lost(libs, "feed_forward" if dtype == BF else "blocks_tc", cta, warp, lambda lib: fn(lib, x, sx, W, sw, y, e))
    assert e.item() == m.DEV_WAIT_TIMEOUT
    assert ((y == want) | (y == OLD)).all()
    e.zero_()
    fn(lost, x, sx, W, sw, y, e)
    assert e.item() == 0 and torch.equal(y, want)


@pytest.mark.parametrize("which", ["feed_forward", "gated_grad"])
@pytest.mark.parametrize("cta, warp", [(1, 5), (0, 9)])
def test_backward_writes_nothing_wrong(libs, which, cta, warp):
    m, lib, lost = libs
    g = gen(4)
    N, d, F = 1500, 512, 640
    x, _, W, _ = inputs(g, BF, N, d, 2 * F, 0)
    dh = randn(g, N, F).to(BF)

    def run(lib):
        e = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = old(N, d), old(2 * F, d), old(N, 2, F)
        call(lib.molora_gated_linear_backward, p(x), 1, N, d, p(W), F, 2, p(dh), p(out[2]), p(out[0]), p(out[1]), p(e))
        return out, e.item()
    want, e = run(lib)
    assert e == 0
    got = []
    with_lost(libs, which, cta, warp, lambda lib: got.extend(run(lib)))
    (out, e) = got
    assert e == m.DEV_WAIT_TIMEOUT
    for w, v in zip(want, out):
        assert ((v == w) | (torch.isnan(v) if which == "feed_forward" else v == OLD)).all()
    if which == "feed_forward":
        assert torch.isnan(out[2]).any() and torch.isnan(out[0]).any() and torch.isnan(out[1]).any()
    out, e = run(lost)
    assert e == 0 and all(torch.equal(w, v) for w, v in zip(want, out))


@pytest.mark.parametrize("which", ["feed_forward", "gated_grad"])
@pytest.mark.parametrize("cta, warp", [(1, 5), (0, 9), (0, 0)])
def test_few_tokens_backward_loses_to_nan(libs, which, cta, warp):
    """Few tokens' dx is a product of its own (csrc/feed_forward.cu), which makes NaN of what it loses."""
    m, lib, lost = libs
    g = gen(5)
    N, d, F = 64, 512, 2048
    x, _, W, _ = inputs(g, BF, N, d, 2 * F, 0)
    dh = randn(g, N, F).to(BF)

    def run(lib):
        e = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = old(N, d), old(2 * F, d), old(N, 2, F)
        call(lib.molora_gated_linear_backward, p(x), 1, N, d, p(W), F, 2, p(dh), p(out[2]), p(out[0]), p(out[1]), p(e))
        return out, e.item()
    want, e = run(lib)
    assert e == 0
    got = []
    with_lost(libs, which, cta, warp, lambda lib: got.extend(run(lib)))
    (out, e) = got
    assert e == m.DEV_WAIT_TIMEOUT
    if which == "gated_grad":  # dW's alone
        assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2]) and ((out[1] == want[1]) | (out[1] == OLD)).all()
    else:
        assert all(((v == w) | torch.isnan(v)).all() for w, v in zip(want, out)) and torch.isnan(out[0]).any()
    out, e = run(lost)
    assert e == 0 and all(torch.equal(w, v) for w, v in zip(want, out))


@pytest.mark.parametrize("cta, warp", [(0, 0), (1, 5), (0, 9)])
def test_chains_of_long_sums_write_nothing_wrong(libs, cta, warp):
    """Sums of several chains of K blocks (over 9000 tokens, and over 2 x 4200 columns): a lost chain is a lost tile."""
    m, lib, lost = libs
    g = gen(6)
    N, d, F = 9000, 256, 4200
    x, _, W, _ = inputs(g, BF, N, d, 2 * F, 0)
    dh = randn(g, N, F).to(BF)

    def run(lib):
        e = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = old(N, d), old(2 * F, d), old(N, 2, F)
        call(lib.molora_gated_linear_backward, p(x), 1, N, d, p(W), F, 2, p(dh), p(out[2]), p(out[0]), p(out[1]), p(e))
        return out, e.item()
    want, e = run(lib)
    assert e == 0
    got = []
    with_lost(libs, "gated_grad", cta, warp, lambda lib: got.extend(run(lib)))
    (out, e) = got
    assert e == m.DEV_WAIT_TIMEOUT
    assert all(((v == w) | (v == OLD)).all() for w, v in zip(want, out))
    out, e = run(lost)
    assert e == 0 and all(torch.equal(w, v) for w, v in zip(want, out))


@pytest.mark.parametrize("cta, warp", [(0, 0), (1, 5), (0, 9)])
def test_chains_of_wide_inputs_write_nothing_wrong(libs, cta, warp):
    """Projections of several chains of K blocks: a lost chain is a lost tile, of h as it was, of dproj NaN."""
    m, lib, lost = libs
    g = gen(7)
    N, d, F = 9000, 8400, 264
    x, _, W, _ = inputs(g, BF, N, d, 2 * F, 0)
    dh = randn(g, N, F).to(BF)

    def run(lib):
        e = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = old(N, F), old(N, 2, F)
        gated(lib, x, None, W, None, out[0], e)
        call(lib.molora_gated_linear_backward, p(x), 1, N, d, p(W), F, 2, p(dh), p(out[1]), None, None, p(e))
        return out, e.item()
    want, e = run(lib)
    assert e == 0
    got = []
    with_lost(libs, "feed_forward", cta, warp, lambda lib: got.extend(run(lib)))
    (out, e) = got
    assert e == m.DEV_WAIT_TIMEOUT
    assert ((out[0] == want[0]) | (out[0] == OLD)).all() and ((out[1] == want[1]) | torch.isnan(out[1])).all()
    assert (out[0] != want[0]).any() and torch.isnan(out[1]).any()
    out, e = run(lost)
    assert e == 0 and all(torch.equal(w, v) for w, v in zip(want, out))
