"""The norm, the expert gate, the base product and the adapted projection refuse bad arguments before
anything is launched: in the binding (ValueError, on CPU tensors) and in the C ABI (status codes)."""

import ctypes
import shutil

import pytest
import torch

import token_adapter_routing_gb300 as m

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not available")

BF, F32, FP8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


SHARED = z(4, 8)


@pytest.mark.parametrize("kwargs, match", [
    (dict(x=z(4)), "x must be a 2-D tensor"),
    (dict(x=z(4, 0)), "at least one column"),
    (dict(x=z(4, 8, dtype=torch.float16)), "x must be one of"),
    (dict(weight=z(7)), "weight must have shape"),
    (dict(weight=z(8, dtype=F32)), "weight must be torch.bfloat16"),
    (dict(residual=z(4, 7)), "residual must have shape"),
    (dict(eps=0.0), "eps"),
    (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"),
    (dict(out8=z(4, 8, dtype=FP8)), "go together"),
    (dict(scale8=z(4, dtype=F32)), "go together"),
    (dict(sum_out=z(4, 8)), "needs a residual"),
    (dict(residual=z(4, 8), sum_out=SHARED, out=SHARED), "different tensors"),
    (dict(x=z(8, 4).t()), "x must be contiguous"),
    (dict(), "must be a CUDA tensor"),
])
def test_rmsnorm_refuses(kwargs, match):
    args = dict(x=z(4, 8), weight=z(8)) | kwargs
    with pytest.raises(ValueError, match=match):
        m.molora_rmsnorm(**args)


@pytest.mark.parametrize("kwargs, match", [
    (dict(logits=z(8)), "2-D"),
    (dict(logits=z(4, 520)), "at most 512"),
    (dict(logits=z(4, 8, dtype=I32)), "must be one of"),
    (dict(score="tanh"), "score must be one of"),
    (dict(groups=3), "groups must be"),
    (dict(groups=0), "groups must be"),
    (dict(groups=4, keep_groups=5), "keep_groups"),
    (dict(groups=4, keep_groups=0), "keep_groups"),
    (dict(groups=8, group_top=2, keep_groups=8), "group_top"),
    (dict(group_top=3), "group_top"),
    (dict(k=0), "k must be"),
    (dict(k=9), "k must be"),
    (dict(groups=4, keep_groups=1, k=3), "k must be"),
    (dict(bias=z(7, dtype=F32)), "bias must have shape"),
    (dict(bias=z(8)), "bias must be torch.float32"),
    (dict(), "must be a CUDA tensor"),
])
def test_gate_refuses(kwargs, match):
    args = dict(logits=z(4, 8), k=2) | kwargs
    with pytest.raises(ValueError, match=match):
        m.molora_gate_topk(**args)


@pytest.mark.parametrize("kwargs, match", [
    (dict(x=z(4, 8, dtype=torch.float16)), "x must be one of"),
    (dict(W=z(6, 7)), "W must have shape"),
    (dict(W=z(6, 8, dtype=F32)), "W must be torch.bfloat16"),
    (dict(W=z(0, 8)), "W must be"),
    (dict(act="tanh"), "act must be one of"),
    (dict(x_scale=z(4, dtype=F32)), "x_scale and w_scale"),
    (dict(x=z(4, 8, dtype=FP8), W=z(6, 8, dtype=FP8)), "x_scale and w_scale"),
    (dict(bias=z(5, dtype=F32)), "bias must have shape"),
    (dict(bias=z(6)), "bias must be torch.float32"),
    (dict(y=z(4, 6, dtype=torch.float16)), "y must be"),
    (dict(out_dtype=torch.float16), "out_dtype must be"),
    (dict(out_dtype=torch.float64), "out_dtype must be"),
    (dict(y=z(4, 6), residual=z(4, 6, dtype=F32)), "residual must be torch.bfloat16"),
    (dict(y=z(4, 6), residual=z(3, 6)), "residual must have shape"),
    (dict(), "must be a CUDA tensor"),
])
def test_linear_refuses(kwargs, match):
    args = dict(x=z(4, 8), W=z(6, 8)) | kwargs
    with pytest.raises(ValueError, match=match):
        m.molora_linear(**args)


@pytest.mark.parametrize("kwargs, match", [
    (dict(W=z(6, 8, dtype=F32)), "W must be"),
    (dict(W=z(6, 8, dtype=FP8)), "w_scale is needed"),
    (dict(h8=z(4, 8, dtype=FP8)), "w_scale is needed"),
    (dict(A=z(2, 8)), "A must be"),
    (dict(A=z(2, 7, 16)), "A must have shape"),
    (dict(B=z(2, 16, 5)), "B must have shape"),
    (dict(ids=z(3, dtype=I32)), "ids must be"),
    (dict(w=z(4, 2, dtype=F32)), "w must have shape"),
    (dict(y=z(4, 6, dtype=torch.float16)), "y must be"),
    (dict(sum_out=z(4, 8)), "needs a residual"),
    (dict(eps=-1.0), "eps"),
    (dict(), "must be a CUDA tensor"),
])
def test_adapted_projection_refuses(kwargs, match):
    args = dict(x=z(4, 8), norm_weight=z(8), eps=1e-6, W=z(6, 8), A=z(2, 8, 16), B=z(2, 16, 6), ids=z(4, dtype=I32),
                y=z(4, 6), scale=1.0) | kwargs
    with pytest.raises(ValueError, match=match):
        m.molora_norm_linear_lora_apply(**args)


@needs_nvcc
def test_c_abi_refuses_without_launching():
    from token_adapter_routing_gb300 import build
    build.build()
    lib = m.load_library()
    p, q, INVALID = 0x10000, 0x20000, 1  # never dereferenced: validation fails first
    norm = lib.molora_rmsnorm
    assert norm(None, 1, 0, 8, None, None, None, 1e-6, None, None, None, None) == 0
    assert norm(p, 2, 4, 8, None, None, p, 1e-6, q, None, None, None) == INVALID      # e4m3 x
    assert norm(p, 1, -1, 8, None, None, p, 1e-6, q, None, None, None) == INVALID
    assert norm(p, 1, 4, 0, None, None, p, 1e-6, q, None, None, None) == INVALID
    assert norm(p, 1, 4, 8, None, None, None, 1e-6, q, None, None, None) == INVALID
    assert norm(p, 1, 4, 8, None, None, p, 0.0, q, None, None, None) == INVALID
    assert norm(p, 1, 4, 8, None, None, p, float("nan"), q, None, None, None) == INVALID
    assert norm(p, 1, 4, 8, None, None, p, 1e-6, None, None, None, None) == INVALID   # no output
    assert norm(p, 1, 4, 8, None, None, p, 1e-6, None, q, None, None) == INVALID      # out8 without scale8
    assert norm(p, 1, 4, 8, None, q, p, 1e-6, q, None, None, None) == INVALID         # sum_out without residual
    assert norm(p, 1, 4, 8, p, q, p, 1e-6, q, None, None, None) == INVALID            # sum_out and out the same
    assert norm(p + 1, 1, 4, 8, None, None, p, 1e-6, q, None, None, None) == INVALID  # half an element
    assert norm(p, 0, 4, 8, None, None, p, 1e-6, q + 2, None, None, None) == INVALID
    most = 2 ** 31 - 1024
    assert norm(p, 1, most + 1, 8, None, None, p, 1e-6, q, None, None, None) == INVALID
    assert norm(p, 1, 1, most + 1, None, None, p, 1e-6, q, None, None, None) == INVALID
    # outputs that share memory with an input in part, with one another, or with the weight
    for bad in [dict(out=p + 16), dict(out=p + 62, residual=q), dict(sum_out=q + 16), dict(out=0x40000), dict(out=0x40000 - 62),
                dict(out8=p), dict(out8=p + 63), dict(out8=q), dict(out8=0x50000), dict(out8=0x50000 - 31), dict(out8=0x4000c),
                dict(scale8=0x30010), dict(scale8=p), dict(sum_out=0x50010), dict(sum_out=0x60000), dict(sum_out=0x30010)]:
        a = dict(x=p, residual=q, sum_out=q, weight=0x40000, out=0x50000, out8=0x30000, scale8=0x60000) | bad
        assert norm(a["x"], 1, 4, 8, a["residual"], a["sum_out"], a["weight"], 1e-6, a["out"], a["out8"], a["scale8"], None) == INVALID, bad
    gate = lib.molora_gate_topk
    assert gate(None, 1, 0, 8, 0, None, 1, 1, 1, 2, 1, 1.0, None, None, None, None) == 0
    for bad in [dict(K=513), dict(K=0), dict(score=2), dict(groups=3), dict(groups=64, K=512), dict(keep=2),
                dict(groups=4, keep=0), dict(top=3), dict(groups=8, top=2), dict(k=0), dict(k=9), dict(k=33, K=64),
                dict(scale=float("nan")), dict(dtype=2), dict(logits=None), dict(ids=None), dict(logits=p + 1),
                dict(ids=p + 2), dict(ids=p + 60), dict(ids=q + 28), dict(logits=q + 16)]:
        a = dict(logits=p, dtype=1, N=4, K=8, score=0, groups=1, keep=1, top=1, k=2, scale=1.0, ids=0x30000) | bad
        assert gate(a["logits"], a["dtype"], a["N"], a["K"], a["score"], None, a["groups"], a["keep"], a["top"], a["k"], 1,
                    a["scale"], a["ids"], q, None, None) == INVALID, bad
    linear = lib.molora_linear
    assert linear(None, 1, None, 0, 8, None, None, 8, None, 0, None, None, 0, None, None) == 0
    for bad in [dict(dtype=3), dict(N=-1), dict(d_in=0), dict(d_out=0), dict(act=5), dict(act=-1), dict(x=None),
                dict(W=None), dict(y=None), dict(sx=p), dict(sw=p), dict(dtype=2), dict(dtype=2, sx=p), dict(x=p + 1),
                dict(y=q + 2), dict(dtype=2, sx=p + 1, sw=p), dict(N=most + 1), dict(d_in=most + 1), dict(d_out=most + 1),
                dict(y=p), dict(y=p + 60), dict(y=p - 124), dict(y=0x30040), dict(bias=q + 124), dict(bias=q - 28),
                dict(res=q + 4), dict(res=q - 124), dict(dtype=2, sx=q + 16, sw=p), dict(dtype=2, sx=p, sw=q - 16)]:
        a = dict(x=p, dtype=1, sx=None, N=4, d_in=8, W=0x30000, sw=None, d_out=8, bias=None, act=0, res=None, y=q) | bad
        assert linear(a["x"], a["dtype"], a["sx"], a["N"], a["d_in"], a["W"], a["sw"], a["d_out"], a["bias"], a["act"], a["res"],
                      a["y"], 0, None, None) == INVALID, bad
    step = lib.molora_norm_linear_lora_apply
    size = ctypes.c_size_t(99)
    for bad in [dict(w_dtype=0), dict(w_dtype=2), dict(h=None), dict(h8=p), dict(W=None), dict(A=None), dict(ids=None),
                dict(k=3), dict(r=12), dict(y=0x10004), dict(eps=0.0), dict(sum_out=q), dict(ws=0x10001),
                dict(h=q), dict(W=q + 64), dict(A=q + 1020), dict(B=q - 4094)]:
        a = dict(w_dtype=1, h=0x30000, h8=None, W=p, A=p, B=p, ids=p, k=1, r=16, y=q, eps=1e-6, sum_out=None, ws=None) | bad
        assert step(p, 1, 4, 64, None, a["sum_out"], p, a["eps"], a["h"], a["h8"], None, a["W"], a["w_dtype"], None, 64, None,
                    a["A"], a["B"], 2, a["r"], a["ids"], None, a["k"], None, None, None, 1.0, a["y"], 0, a["ws"],
                    ctypes.byref(size) if a["ws"] else None, None, None) == INVALID, bad
