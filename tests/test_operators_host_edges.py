"""The adapted projection refuses outputs over what is still to be read, and takes its slots in the shapes that the apply
takes."""

import ctypes
import shutil

import pytest
import torch

import token_adapter_routing_gb300 as m

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not available")

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32

# N = 4, d_in = 64, d_out = 32, K = 2, r = 16, k = 2, e4m3 W: the arrays one after another, with room between
SIZES = dict(x=512, residual=512, sum_out=512, norm_weight=128, h=512, h8=256, scale8=16, W=2048, w_scale=128, bias=128,
             A=4096, B=2048, ids=32, w=32, counts=8, offsets=12, perm=32, y=512, ws=4096)
PLACES = {name: 0x100000 + 0x10000 * i for i, name in enumerate(SIZES)}


def step(**at):
    a = PLACES | at
    size = ctypes.c_size_t(SIZES["ws"])
    return m.load_library().molora_norm_linear_lora_apply(
        a["x"], 1, 4, 64, a["residual"], a["sum_out"], a["norm_weight"], 1e-6, a["h"], a["h8"], a["scale8"], a["W"], 2,
        a["w_scale"], 32, a["bias"], a["A"], a["B"], 2, 16, a["ids"], a["w"], 2, a["counts"], a["offsets"], a["perm"], 1.0,
        a["y"], 0, a["ws"], ctypes.byref(size), None, None)


@needs_nvcc
@pytest.mark.parametrize("read", ["W", "w_scale", "bias", "A", "B", "ids", "w", "counts", "offsets", "perm"])
@pytest.mark.parametrize("written", ["sum_out", "h", "h8", "scale8", "y", "ws"])
def test_outputs_over_what_is_still_read(written, read):
    from token_adapter_routing_gb300 import build
    build.build()
    # the output's first bytes in the array's last ones, on a boundary that every check before allows
    place = PLACES[read] + SIZES[read] - 4
    place -= place % {"h": 16, "y": 16, "sum_out": 2, "ws": 256}.get(written, 4)
    assert step(**{written: place}) == 1


@needs_nvcc
@pytest.mark.parametrize("one, other", [("ws", "h"), ("ws", "h8"), ("ws", "scale8"), ("ws", "y")])
def test_workspace_over_an_output(one, other):
    from token_adapter_routing_gb300 import build
    build.build()
    assert step(**{other: PLACES[one] + 64}) == 1


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("kwargs", [
    dict(ids=z(4, 1, dtype=I32)), dict(w=z(4, 1, dtype=F32)), dict(ids=z(4, 1, dtype=I32), w=z(4, dtype=F32)),
    dict(ids=z(4, 2, dtype=I32), w=z(4, 2, dtype=F32), counts=z(2, dtype=I32), offsets=z(3, dtype=I32), perm=z(4, 2, dtype=I32)),
    dict(counts=z(2, 1, dtype=I32), offsets=z(1, 3, dtype=I32), perm=z(4, 1, dtype=I32))])
def test_slots_in_the_shapes_that_the_apply_takes(kwargs):
    """molora_lora_apply takes these: the one reason left to refuse them is that they are on the CPU."""
    args = dict(x=z(4, 8), norm_weight=z(8), eps=1e-6, W=z(6, 8), A=z(2, 8, 16), B=z(2, 16, 6), ids=z(4, dtype=I32),
                y=z(4, 6), scale=1.0) | kwargs
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        m.molora_norm_linear_lora_apply(**args)


@pytest.mark.parametrize("kwargs, match", [
    (dict(w=z(2, 2, dtype=F32)), "w must have shape"), (dict(w=z(4, 1)), "w must be torch.float32"),
    (dict(counts=z(3, dtype=I32)), "counts must have shape"), (dict(perm=z(5, dtype=I32)), "perm must have shape"),
    (dict(offsets=z(3, dtype=F32)), "offsets must be torch.int32")])
def test_slots_of_other_sizes_are_refused(kwargs, match):
    args = dict(x=z(4, 8), norm_weight=z(8), eps=1e-6, W=z(6, 8), A=z(2, 8, 16), B=z(2, 16, 6), ids=z(4, dtype=I32),
                y=z(4, 6), scale=1.0) | kwargs
    with pytest.raises(ValueError, match=match):
        m.molora_norm_linear_lora_apply(**args)
