"""The block-scaled product, its quantiser and the gated feed-forward block refuse bad arguments before anything is
launched: in the binding (ValueError, on CPU tensors) and in the C ABI (status codes)."""

import shutil

import pytest
import torch

import token_adapter_routing_gb300 as m

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not available")

BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("kwargs, match", [
    (dict(x=z(4)), "x must be a 2-D tensor"),
    (dict(x=z(4, 0)), "at least one column"),
    (dict(x=z(4, 8, dtype=FP8)), "x must be one of"),
    (dict(x=z(200, 4).t()), "x must be contiguous"),
    (dict(out8=z(4, 200)), "out8 must be torch.float8"),
    (dict(out8=z(4, 199, dtype=FP8)), "out8 must have shape"),
    (dict(scale8=z(4, 1, dtype=F32)), "scale8 must have shape"),
    (dict(scale8=z(4, 2)), "scale8 must be torch.float32"),
    (dict(), "must be a CUDA tensor"),
])
def test_quantise_refuses(kwargs, match):
    with pytest.raises(ValueError, match=match):
        m.molora_quantise_blocks(**(dict(x=z(4, 200)) | kwargs))


@pytest.mark.parametrize("kwargs, match", [
    (dict(x=z(4, 160)), "x must be one of"),
    (dict(W=z(150, 144, dtype=FP8)), "W must have shape"),
    (dict(W=z(150, 160)), "W must be torch.float8"),
    (dict(W=z(0, 160, dtype=FP8)), "W must be"),
    (dict(x_scale=None), "must be tensors"),
    (dict(w_scale=None), "must be tensors"),
    (dict(x_scale=z(4, 1, dtype=F32)), "x_scale must have shape"),
    (dict(x_scale=z(4, dtype=F32)), "x_scale must have shape"),
    (dict(w_scale=z(1, 2, dtype=F32)), "w_scale must have shape"),
    (dict(w_scale=z(150, 2, dtype=F32)), "w_scale must have shape"),
    (dict(w_scale=z(2, 2)), "w_scale must be torch.float32"),
    (dict(act="tanh"), "act must be one of"),
    (dict(bias=z(149, dtype=F32)), "bias must have shape"),
    (dict(y=z(4, 150, dtype=torch.float16)), "y must be"),
    (dict(out_dtype=torch.float16), "out_dtype must be"),
    (dict(residual=z(4, 150)), "residual must be torch.float32"),
    (dict(), "must be a CUDA tensor"),
])
def test_linear_blocks_refuses(kwargs, match):
    args = dict(x=z(4, 160, dtype=FP8), x_scale=z(4, 2, dtype=F32), W=z(150, 160, dtype=FP8), w_scale=z(2, 2, dtype=F32)) | kwargs
    with pytest.raises(ValueError, match=match):
        m.molora_linear_blocks(**args)


@pytest.mark.parametrize("kwargs, match", [
    (dict(x=z(4, 16, dtype=F32)), "x must be one of"),
    (dict(W=z(11, 16)), "W must be a 2-D"),
    (dict(W=z(12, 8)), "W must have shape"),
    (dict(W=z(12, 16, dtype=F32)), "W must be torch.bfloat16"),
    (dict(act="swish"), "act must be one of"),
    (dict(h=z(4, 12)), "h must have shape"),
    (dict(h=z(4, 6, dtype=F32)), "h must be torch.bfloat16"),
    (dict(x_scale=z(4, 1, dtype=F32)), "x_scale and w_scale"),
    (dict(x=z(4, 16, dtype=FP8), W=z(12, 16, dtype=FP8)), "x_scale and w_scale"),
    (dict(x=z(4, 16, dtype=FP8), W=z(12, 16, dtype=FP8), x_scale=z(4, 1, dtype=F32), w_scale=z(1, 1, dtype=F32)), "w_scale must have shape"),
    (dict(), "must be a CUDA tensor"),
])
def test_gated_refuses(kwargs, match):
    with pytest.raises(ValueError, match=match):
        m.molora_gated_linear(**(dict(x=z(4, 16), W=z(12, 16)) | kwargs))


@pytest.mark.parametrize("kwargs, match", [
    (dict(x=z(4, 16, dtype=FP8)), "x must be one of"),
    (dict(W=z(13, 16)), "W must be a 2-D"),
    (dict(dh=None), "must be a tensor"),
    (dict(dh=z(4, 8)), "dh must have shape"),
    (dict(dh=z(4, 6, dtype=F32)), "dh must be torch.bfloat16"),
    (dict(dx=z(4, 8)), "dx must have shape"),
    (dict(dW=z(6, 16)), "dW must have shape"),
    (dict(dW=z(12, 16, dtype=F32)), "dW must be torch.bfloat16"),
    (dict(dproj=z(4, 2, 7)), "dproj must have shape"),
    (dict(act="tanh"), "act must be one of"),
    (dict(), "must be a CUDA tensor"),
])
def test_gated_backward_refuses(kwargs, match):
    with pytest.raises(ValueError, match=match):
        m.molora_gated_linear_backward(**(dict(x=z(4, 16), W=z(12, 16), dh=z(4, 6)) | kwargs))


OK, INVALID, UNSUPPORTED = 0, 1, 2
F, B, Q = 0, 1, 2
X, WT, SX, SW, Y, R, P, BIAS = (0x100000 * i for i in range(1, 9))  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from token_adapter_routing_gb300 import build
    build.build()
    return m.load_library()


@needs_nvcc
def test_c_abi_quantise(lib):
    f = lib.molora_quantise_blocks
    assert f(X, B, 0, 128, None, None, None) == OK
    for bad in [(X, Q, 4, 128, Y, SX), (X, B, -1, 128, Y, SX), (X, B, 4, 0, Y, SX), (None, B, 4, 128, Y, SX), (X, B, 4, 128, None, SX),
                (X, B, 4, 128, Y, None), (X + 1, B, 4, 128, Y, SX), (X + 2, F, 4, 128, Y, SX), (X, B, 4, 128, Y, SX + 2),
                (X, B, 4, 128, X + 64, SX), (X, B, 4, 128, Y, Y + 256), (X, B, 4, 128, Y, X), (X, B, 2 ** 31, 128, Y, SX),
                (X, B, 4, 2 ** 31 - 1000, Y, SX)]:
        assert f(*bad, None) == INVALID, bad


@needs_nvcc
def test_c_abi_linear_blocks(lib):
    f = lib.molora_linear_blocks
    good = dict(x=X, sx=SX, N=4, d_in=160, W=WT, sw=SW, d_out=150, bias=None, act=0, res=None, y=Y, y16=0)

    def call(**kw):
        return f(*(good | kw).values(), None, None)
    assert call(N=0, x=None, W=None, y=None) == OK
    for bad in [dict(N=-1), dict(d_in=0), dict(d_out=0), dict(act=5), dict(act=-1), dict(x=None), dict(W=None), dict(y=None),
                dict(sx=None), dict(sw=None), dict(x=X + 8), dict(W=WT + 1), dict(sx=SX + 2), dict(sw=SW + 1), dict(bias=BIAS + 2),
                dict(y=Y + 2), dict(y=Y + 1, y16=1), dict(res=R + 2), dict(y=X), dict(y=WT + 16), dict(y=SX + 8), dict(y=SW),
                dict(bias=Y + 32), dict(res=Y + 16), dict(N=2 ** 31 - 1000), dict(d_out=2 ** 31 - 1000)]:
        assert call(**bad) == INVALID, bad
    assert call(d_in=168) == UNSUPPORTED and call(d_in=1) == UNSUPPORTED and call(N=0, d_in=24) == UNSUPPORTED


@needs_nvcc
def test_c_abi_gated(lib):
    f = lib.molora_gated_linear
    good = dict(x=X, dtype=B, sx=None, N=4, d_in=64, W=WT, sw=None, d_ff=50, act=2, h=Y)

    def call(**kw):
        return f(*(good | kw).values(), None, None)
    fp8 = dict(dtype=Q, sx=SX, sw=SW)
    assert call(N=0, x=None, W=None, h=None) == OK and call(N=0, **fp8) == OK
    for bad in [dict(dtype=F), dict(dtype=3), dict(N=-1), dict(d_in=0), dict(d_ff=0), dict(act=9), dict(x=None), dict(W=None),
                dict(h=None), dict(sx=SX), dict(sw=SW), dict(x=X + 2), dict(W=WT + 8), dict(h=Y + 1), dict(h=X),
                dict(h=WT + 2 * 99 * 64), dict(d_ff=2 ** 30), fp8 | dict(sx=None), fp8 | dict(sw=None), fp8 | dict(h=SX), fp8 | dict(h=SW)]:
        assert call(**bad) == INVALID, bad
    assert call(d_in=63) == UNSUPPORTED and call(d_in=4) == UNSUPPORTED and call(**(fp8 | dict(d_in=72))) == UNSUPPORTED


@needs_nvcc
def test_c_abi_gated_backward(lib):
    f = lib.molora_gated_linear_backward
    good = dict(x=X, dtype=B, N=4, d_in=64, W=WT, d_ff=50, act=2, dh=SX, dproj=P, dx=Y, dW=R)

    def call(**kw):
        return f(*(good | kw).values(), None, None)
    assert call(N=0, x=None, W=None, dh=None, dproj=None, dx=None, dW=None) == OK
    for bad in [dict(dtype=F), dict(dtype=Q), dict(N=-1), dict(d_in=0), dict(d_ff=0), dict(act=5), dict(x=None), dict(W=None),
                dict(dh=None), dict(dproj=None), dict(x=X + 2), dict(W=WT + 2), dict(dproj=P + 2), dict(dx=Y + 8), dict(dW=R + 2), dict(dh=SX + 1), dict(dx=X), dict(dx=P), dict(dW=WT), dict(dW=X), dict(dx=SX),
                dict(dproj=SX), dict(dproj=X), dict(dproj=WT), dict(dx=R), dict(dW=Y), dict(dproj=Y), dict(dproj=R + 128)]:
        assert call(**bad) == INVALID, bad
    assert call(d_in=60) == UNSUPPORTED and call(N=0, d_in=60) == UNSUPPORTED
