"""Python binding of the GB300 per-token adapter routing library (include/molora.h).

Argument marshalling only: every function here checks the shapes, dtypes and devices of
torch CUDA tensors against the sizes the call implies, passes their device pointers and
the tensors' current CUDA stream through ctypes to the C ABI, and raises on a non-OK
status.  A mis-sized tensor raises ValueError before anything is launched.  All
computation happens in the library's CUDA kernels; there is no CPU or PyTorch fallback.  If
the compiled library is missing the first call raises: build it with
``token_adapter_routing_gb300.build.build()``.

Method: "MoLoRA: Composable Specialization via Per-Token Adapter Routing" -- vocabulary
routing and the learned top-k router (Table 1), dispatch by histogram / pointer arrays /
grouping (Table 1, Figure 2), and the batched LoRA apply over a GPU-resident hot set
(Figure 2, Figure 4, Table 10 shapes).
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch

from . import build as _build

__all__ = [
    "molora_route_vocab", "molora_router_topk", "molora_dispatch", "molora_route_vocab_dispatch",
    "molora_lora_apply", "molora_lora_apply_masked_pass", "molora_route_vocab_lora_apply",
    "molora_router_lora_apply", "molora_rmsnorm", "molora_gate_topk", "molora_linear",
    "molora_norm_linear_lora_apply", "molora_quantise_blocks", "molora_linear_blocks", "molora_gated_linear",
    "molora_gated_linear_backward", "molora_select_path", "molora_workspace_bytes", "molora_lora_apply_static_ws",
    "molora_selftest_bounded_wait", "library_path", "load_library",
    "MoloraError", "PATHS", "DEV_TOKEN_OUTSIDE_RANGES", "DEV_BAD_RANGES", "DEV_BAD_ADAPTER_ID",
    "DEV_BAD_PERMUTATION", "DEV_WAIT_TIMEOUT", "DEV_BAD_LOGIT", "MAX_ADAPTERS", "MAX_EXPERTS", "MAX_GATE_K",
    "MAX_GROUPS", "SCALE_BLOCK", "ROUTER_HIDDEN", "ACTIVATIONS", "SCORES",
]

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_SCRATCH_TOO_SMALL = 0, 1, 2, 3, 4
STATIC_SCRATCH_BYTES = 16 << 20
F32, BF16, E4M3 = 0, 1, 2
PATHS = {"auto": 0, "scalar": 1, "grouped": 2, "dense": 3, "stacked": 4}
PATH_NAMES = {v: k for k, v in PATHS.items()}
DEV_TOKEN_OUTSIDE_RANGES = 0x1
DEV_BAD_RANGES = 0x2
DEV_BAD_ADAPTER_ID = 0x4
DEV_BAD_PERMUTATION = 0x8
DEV_WAIT_TIMEOUT = 0x10
DEV_BAD_LOGIT = 0x20
INPUTS_READY = 0x1  # molora_route_vocab_dispatch_ex flag
MAX_ADAPTERS = 64
MAX_EXPERTS, MAX_GATE_K, MAX_GROUPS = 512, 32, 32
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
SCORES = {"softmax": 0, "sigmoid": 1}
ROUTER_HIDDEN = 64
SCALE_BLOCK = 128  # columns (and, of weights, rows) that share a scale in the block-scaled calls

EXPORTED = ("molora_route_vocab", "molora_route_vocab_ex", "molora_router_topk", "molora_dispatch", "molora_route_vocab_dispatch",
            "molora_route_vocab_dispatch_ex", "molora_route_vocab_lora_apply_ex",
            "molora_lora_apply", "molora_router_lora_apply", "molora_route_vocab_lora_apply",
            "molora_lora_apply_ex", "molora_lora_apply_bf16y", "molora_lora_apply_indirect",
            "molora_lora_apply_masked_pass", "molora_select_path", "molora_status_string", "molora_version",
            "molora_selftest_bounded_wait", "molora_lora_apply_static_ws", "molora_rmsnorm", "molora_gate_topk",
            "molora_linear", "molora_norm_linear_lora_apply", "molora_quantise_blocks", "molora_linear_blocks",
            "molora_gated_linear", "molora_gated_linear_backward")


class MoloraError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


_lib = None


def library_path() -> str:
    return _build.LIB


def load_library(path=None):
    """Loads the compiled library (raises if it has not been built).  ``path``: another build of
    it (the tuning build of build.build(tuning=True)); only the first load in a process counts."""
    global _lib
    if _lib is not None:
        if path is not None and os.path.realpath(path) != os.path.realpath(_lib._name):
            raise RuntimeError(f"a different CUDA library ({_lib._name}) is already loaded")
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is missing: build it with token_adapter_routing_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I64, I32, F, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_int
    lib.molora_route_vocab.argtypes = [P, I64, P, I32, P, P, P]
    lib.molora_route_vocab_ex.argtypes = [P, I64, P, I32, P, P, ctypes.c_uint32, P]
    lib.molora_router_topk.argtypes = [P, S, I64, I32, P, P, P, P, I32, I32, P, P, P, P]
    lib.molora_dispatch.argtypes = [P, I64, I32, I32, P, P, P, P, P]
    lib.molora_route_vocab_dispatch.argtypes = [P, I64, P, I32, P, P, P, P, P, P]
    lib.molora_route_vocab_dispatch_ex.argtypes = [P, I64, P, I32, P, P, P, P, P, ctypes.c_uint32, P]
    lib.molora_lora_apply.argtypes = [P, S, I64, I32, I32, P, P, I32, I32, P, P, I32, P, P, P, F, P, P, P, P, P]
    lib.molora_lora_apply_ex.argtypes = [P, S, I64, I32, I32, P, P, I32, I32, P, P, I32, P, P, P, F, P, P, P, P, S,
                                         P]
    lib.molora_lora_apply_bf16y.argtypes = [P, S, I64, I32, I32, P, P, I32, I32, P, P, I32, P, P, P, F, P, P, S, P]
    lib.molora_lora_apply_indirect.argtypes = [P, S, I64, I32, I32, P, P, I32, I32, P, P, I32, P, P, P, F, P, I32,
                                               P, S, P]
    lib.molora_router_lora_apply.argtypes = [P, S, I64, I32, I32, P, P, P, P, P, P, I32, I32, I32, F, P, P, P, P,
                                             I32, P, P, P, P]
    lib.molora_route_vocab_lora_apply.argtypes = [P, I64, P, I32, P, S, I32, I32, P, P, I32, F, P, I32, P, P, P, P,
                                                  P, P]
    lib.molora_route_vocab_lora_apply_ex.argtypes = [P, I64, P, I32, P, S, I32, I32, P, P, I32, F, P, I32, P, P, P,
                                                     P, P, ctypes.c_uint32, P]
    lib.molora_lora_apply_masked_pass.argtypes = [P, S, I64, I32, I32, P, P, I32, I32, P, I32, F, P, P, S, P]
    lib.molora_lora_apply_static_ws.argtypes = [P, S, I64, I32, I32, P, P, I32, I32, P, P, I32, F, P, P, P]
    lib.molora_rmsnorm.argtypes = [P, S, I64, I32, P, P, P, F, P, P, P, P]
    lib.molora_gate_topk.argtypes = [P, S, I64, I32, S, P, I32, I32, I32, I32, I32, F, P, P, P, P]
    lib.molora_linear.argtypes = [P, S, P, I64, I32, P, P, I32, P, S, P, P, I32, P, P]
    lib.molora_norm_linear_lora_apply.argtypes = [P, S, I64, I32, P, P, P, F, P, P, P, P, S, P, I32, P, P, P, I32, I32,
                                                  P, P, I32, P, P, P, F, P, I32, P, P, P, P]
    lib.molora_quantise_blocks.argtypes = [P, S, I64, I32, P, P, P]
    lib.molora_linear_blocks.argtypes = [P, P, I64, I32, P, P, I32, P, S, P, P, I32, P, P]
    lib.molora_gated_linear.argtypes = [P, S, P, I64, I32, P, P, I32, S, P, P, P]
    lib.molora_gated_linear_backward.argtypes = [P, S, I64, I32, P, I32, S, P, P, P, P, P, P]
    lib.molora_select_path.argtypes = [S, I64, I32, I32, I32, I32, I32]
    lib.molora_status_string.argtypes = [S]
    lib.molora_status_string.restype = ctypes.c_char_p
    lib.molora_version.argtypes = []
    lib.molora_selftest_bounded_wait.argtypes = [ctypes.c_uint32, P, P]
    for name in ("molora_route_vocab", "molora_route_vocab_ex", "molora_router_topk", "molora_dispatch", "molora_route_vocab_dispatch",
                 "molora_route_vocab_dispatch_ex", "molora_route_vocab_lora_apply_ex", "molora_lora_apply", "molora_lora_apply_ex", "molora_lora_apply_bf16y", "molora_lora_apply_indirect",
                 "molora_router_lora_apply", "molora_route_vocab_lora_apply", "molora_lora_apply_masked_pass",
                 "molora_select_path", "molora_version", "molora_selftest_bounded_wait",
                 "molora_lora_apply_static_ws", "molora_rmsnorm", "molora_gate_topk", "molora_linear",
                 "molora_norm_linear_lora_apply", "molora_quantise_blocks", "molora_linear_blocks", "molora_gated_linear",
                 "molora_gated_linear_backward"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != OK:
        raise MoloraError(fn, status, load_library().molora_status_string(status).decode())


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, device) -> ctypes.c_void_p:
    """The given stream, else the current stream of `device` (the tensors' device, which may
    differ from the current device)."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return ctypes.c_void_p(stream.cuda_stream)


def _cuda(t: torch.Tensor, name: str, dtype=None, ndim=None, device=None):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device} (all tensors of a call share one device)")
    return t


def _sized(t: Optional[torch.Tensor], name: str, numel: int, dtype, device, shape=None):
    """A caller-supplied output or index tensor: CUDA, contiguous, the right dtype, device and
    element count (and exact shape when given)."""
    if t is None:
        return None
    _cuda(t, name, dtype, device=device)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return t


def _need(t: Optional[torch.Tensor], name: str, numel: int, rows: Optional[int] = None):
    """Shape-only check of an optional tensor (before any device check, so that a mis-sized
    argument is reported as such): `numel` elements and, when given, `rows` rows."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()} (shape {tuple(t.shape)})")
    if rows is not None and (t.dim() == 0 or t.shape[0] != rows):
        raise ValueError(f"{name} must have {rows} rows, got shape {tuple(t.shape)}")


def _err_word(err_word: Optional[torch.Tensor], device):
    if err_word is None:
        return None
    _cuda(err_word, "err_word", torch.int32, device=device)
    if err_word.numel() < 1:
        raise ValueError("err_word must hold at least one int32")
    return err_word


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise ValueError(f"unsupported dtype {t.dtype}: use bfloat16 or float32")


def _slots(ids: torch.Tensor, N: int, name: str = "ids"):
    """k for ids of shape [N] (k = 1) or [N, k]; raises unless ids has N rows."""
    if ids.dim() not in (1, 2) or ids.shape[0] != N:
        raise ValueError(f"{name} must be [N] or [N, k] with N = {N}, got {tuple(ids.shape)}")
    return 1 if ids.dim() == 1 else ids.shape[1]


def _workspace(ws: Optional[torch.Tensor], device, call, stream=None) -> int:
    """Runs `call(ws_ptr, ws_bytes_ptr)` under the library's workspace convention and returns
    its status: with no caller buffer it first queries the size and, if one is needed,
    allocates it on `device` (torch's caching allocator; inside a CUDA graph capture the
    graph's pool; of `stream`'s memory if given).  An empty buffer (what a size of 0 makes; it has no address, which
    would be a query) is none."""
    size = ctypes.c_size_t(0)
    if ws is None:
        status = call(None, ctypes.byref(size))
        if status != OK:
            return status
        if size.value == 0:
            return call(None, None)
        with torch.cuda.stream(stream):
            ws = torch.empty(size.value, dtype=torch.uint8, device=device)
    else:
        _cuda(ws, "ws", torch.uint8, device=device)
        if ws.numel() == 0:
            return call(None, None)
    size.value = ws.numel()
    return call(_p(ws), ctypes.byref(size))


def _on_tensor_device(fn):
    """Runs a launching call with the device of its first CUDA tensor argument current, so that
    the library launches on the device that holds the tensors (and their stream), whichever
    device the caller has current.  The call itself checks that all tensors share that device."""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        for a in (*args, *kwargs.values()):
            if isinstance(a, (list, tuple)) and a and isinstance(a[0], torch.Tensor):
                a = a[0]
            if isinstance(a, torch.Tensor) and a.is_cuda:
                if a.device.index == torch.cuda.current_device():
                    return fn(*args, **kwargs)
                with torch.cuda.device(a.device):
                    return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return call


def molora_workspace_bytes(N, d_in, d_out, K, r, k, dtype=torch.bfloat16, path="auto", router=False) -> int:
    """Bytes of workspace molora_lora_apply (or, with router=True, molora_router_lora_apply)
    needs for these sizes (a query: nothing is launched).  Allocate them once, e.g. before
    capturing a CUDA graph, and pass the uint8 buffer as ``ws``."""
    size = ctypes.c_size_t(0)
    lib = load_library()
    code = BF16 if dtype == torch.bfloat16 else F32
    if router:
        _check("molora_router_lora_apply", lib.molora_router_lora_apply(
            None, code, N, d_in, d_out, None, None, None, None, None, None, K, r, k, 1.0, None, None, None, None, 0,
            None, ctypes.byref(size), None, None))
    else:
        _check("molora_lora_apply", lib.molora_lora_apply_ex(
            None, code, N, d_in, d_out, None, None, K, r, None, None, k, None, None, None, 1.0, None, None,
            ctypes.byref(size), None, PATHS[path], None))
    return size.value


@_on_tensor_device
def molora_route_vocab(tok, starts, adapter=None, err_word=None, stream=None):
    """adapter[t] = a with starts[a] <= tok[t] < starts[a+1], else -1 (int32 [N])."""
    return _route_vocab(tok, starts, adapter, err_word, stream, None)


@_on_tensor_device
def molora_route_vocab_ex(tok, starts, flags, adapter=None, err_word=None, stream=None):
    """molora_route_vocab with flags (INPUTS_READY: tok and starts are not written by the kernel
    enqueued just before, so each token is routed before waiting on it)."""
    return _route_vocab(tok, starts, adapter, err_word, stream, int(flags))


def _route_vocab(tok, starts, adapter, err_word, stream, flags):
    _need(adapter, "adapter", tok.numel())
    _cuda(tok, "tok", torch.int32, 1)
    dev = tok.device
    _cuda(starts, "starts", torch.int32, 1, device=dev)
    N, K = tok.numel(), starts.numel() - 1
    if adapter is None:
        adapter = torch.empty(N, dtype=torch.int32, device=dev)
    _sized(adapter, "adapter", N, torch.int32, dev)
    args = (_p(tok), N, _p(starts), K, _p(adapter), _p(_err_word(err_word, dev)))
    if flags is None:
        _check("molora_route_vocab", load_library().molora_route_vocab(*args, _stream(stream, dev)))
    else:
        _check("molora_route_vocab_ex", load_library().molora_route_vocab_ex(*args, flags, _stream(stream, dev)))
    return adapter


@_on_tensor_device
def molora_router_topk(x, W1, W2, k, b1=None, b2=None, logits=None, ids=None, w=None, want_logits=True,
                       stream=None):
    """Learned router: returns (logits fp32 [N,K] or None, ids int32 [N,k], w fp32 [N,k])."""
    if x.dim() != 2 or W1.dim() != 2 or W2.dim() != 2:
        raise ValueError("x must be [N, d_in], W1 [d_in, 64] and W2 [64, K]")
    N, d_in = x.shape
    if tuple(W1.shape) != (d_in, ROUTER_HIDDEN) or W2.shape[0] != ROUTER_HIDDEN:
        raise ValueError("W1 must be [d_in, 64] and W2 [64, K]")
    K = W2.shape[1]
    _need(logits, "logits", N * K, rows=N)
    _need(ids, "ids", N * k, rows=N)
    _need(w, "w", N * k, rows=N)
    _need(b1, "b1", ROUTER_HIDDEN)
    _need(b2, "b2", K)
    _cuda(x, "x", None, 2)
    dev = x.device
    _cuda(W1, "W1", x.dtype, 2, device=dev)
    _cuda(W2, "W2", x.dtype, 2, device=dev)
    _sized(b1, "b1", ROUTER_HIDDEN, torch.float32, dev)
    _sized(b2, "b2", K, torch.float32, dev)
    if logits is None and want_logits:
        logits = torch.empty(N, K, dtype=torch.float32, device=dev)
    if ids is None:
        ids = torch.empty(N, k, dtype=torch.int32, device=dev)
    if w is None:
        w = torch.empty(N, k, dtype=torch.float32, device=dev)
    _sized(logits, "logits", N * K, torch.float32, dev)
    _sized(ids, "ids", N * k, torch.int32, dev)
    _sized(w, "w", N * k, torch.float32, dev)
    _check("molora_router_topk", load_library().molora_router_topk(
        _p(x), _dtype_code(x), N, d_in, _p(W1), _p(b1), _p(W2), _p(b2), K, k, _p(logits), _p(ids), _p(w),
        _stream(stream, dev)))
    return logits, ids, w


@_on_tensor_device
def molora_dispatch(ids, K, counts=None, offsets=None, perm=None, err_word=None, stream=None):
    """Histogram, exclusive-scan offsets and stable slot permutation of ids [N] or [N, k]."""
    N = ids.shape[0]
    k = _slots(ids, N)
    _need(counts, "counts", K)
    _need(offsets, "offsets", K + 1)
    _need(perm, "perm", N * k)
    _cuda(ids, "ids", torch.int32)
    dev = ids.device
    if counts is None:
        counts = torch.empty(K, dtype=torch.int32, device=dev)
    if offsets is None:
        offsets = torch.empty(K + 1, dtype=torch.int32, device=dev)
    if perm is None:
        perm = torch.empty(N * k, dtype=torch.int32, device=dev)
    _sized(counts, "counts", K, torch.int32, dev)
    _sized(offsets, "offsets", K + 1, torch.int32, dev)
    _sized(perm, "perm", N * k, torch.int32, dev)
    _check("molora_dispatch", load_library().molora_dispatch(
        _p(ids), N, k, K, _p(counts), _p(offsets), _p(perm), _p(_err_word(err_word, dev)), _stream(stream, dev)))
    return counts, offsets, perm


@_on_tensor_device
def molora_route_vocab_dispatch(tok, starts, adapter=None, counts=None, offsets=None, perm=None, err_word=None,
                                stream=None):
    """molora_route_vocab then molora_dispatch (k = 1) as one kernel: (adapter, counts, offsets, perm)."""
    return _route_vocab_dispatch(tok, starts, adapter, counts, offsets, perm, err_word, stream, None)


@_on_tensor_device
def molora_route_vocab_dispatch_ex(tok, starts, flags, adapter=None, counts=None, offsets=None, perm=None,
                                   err_word=None, stream=None):
    """molora_route_vocab_dispatch with flags (INPUTS_READY: tok and starts are not written by the
    kernel enqueued just before, so the kernel reads them before waiting on it)."""
    return _route_vocab_dispatch(tok, starts, adapter, counts, offsets, perm, err_word, stream, int(flags))


def _route_vocab_dispatch(tok, starts, adapter, counts, offsets, perm, err_word, stream, flags):
    N, K = tok.numel(), starts.numel() - 1
    for name, t, n in (("adapter", adapter, N), ("counts", counts, K), ("offsets", offsets, K + 1), ("perm", perm, N)):
        _need(t, name, n)
    _cuda(tok, "tok", torch.int32, 1)
    dev = tok.device
    _cuda(starts, "starts", torch.int32, 1, device=dev)
    if adapter is None:
        adapter = torch.empty(N, dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty(K, dtype=torch.int32, device=dev)
    if offsets is None:
        offsets = torch.empty(K + 1, dtype=torch.int32, device=dev)
    if perm is None:
        perm = torch.empty(N, dtype=torch.int32, device=dev)
    _sized(adapter, "adapter", N, torch.int32, dev)
    _sized(counts, "counts", K, torch.int32, dev)
    _sized(offsets, "offsets", K + 1, torch.int32, dev)
    _sized(perm, "perm", N, torch.int32, dev)
    args = (_p(tok), N, _p(starts), K, _p(adapter), _p(counts), _p(offsets), _p(perm), _p(_err_word(err_word, dev)))
    if flags is None:
        _check("molora_route_vocab_dispatch", load_library().molora_route_vocab_dispatch(*args, _stream(stream, dev)))
    else:
        _check("molora_route_vocab_dispatch_ex",
               load_library().molora_route_vocab_dispatch_ex(*args, flags, _stream(stream, dev)))
    return adapter, counts, offsets, perm


@_on_tensor_device
def molora_lora_apply(x, A, B, ids, y, scale, w=None, counts=None, offsets=None, perm=None, err_word=None,
                      path="auto", ws=None, stream=None):
    """y[t] += scale * sum_j w[t,j] (x[t] A_{ids[t,j]}) B_{ids[t,j]}, in place on y (fp32, or bf16
    through molora_lora_apply_bf16y).  A and B are the hot-set slabs [K, d_in, r] and
    [K, r, d_out], or lists of K per-adapter tensors [d_in, r] and [r, d_out] (the indirect
    layout, molora_lora_apply_indirect).  ``ws``: an optional uint8 workspace of
    molora_workspace_bytes bytes; without one, a path that needs it gets a fresh buffer."""
    # shapes first: a mis-sized argument raises before anything else is looked at
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D tensor [N, d_in]")
    N, d_in = x.shape
    indirect = isinstance(A, (list, tuple))
    if indirect:
        if not isinstance(B, (list, tuple)) or len(A) != len(B) or not A:
            raise ValueError("indirect layout: A and B must be lists of the same nonzero length")
        K, r, d_out = len(A), A[0].shape[1], B[0].shape[1]
        if any(tuple(a_i.shape) != (d_in, r) for a_i in A) or any(tuple(b_i.shape) != (r, d_out) for b_i in B):
            raise ValueError("indirect layout: every A[i] must be [d_in, r] and every B[i] [r, d_out]")
    else:
        if A.dim() != 3 or B.dim() != 3:
            raise ValueError("A must be [K, d_in, r] and B [K, r, d_out]")
        K, _, r = A.shape
        d_out = B.shape[2]
        if A.shape[1] != d_in or tuple(B.shape[:2]) != (K, r):
            raise ValueError("A must be [K, d_in, r] and B [K, r, d_out]")
    k = _slots(ids, N)
    if y.dim() != 2 or tuple(y.shape) != (N, d_out):
        raise ValueError(f"y must be [N, d_out] = {(N, d_out)}, got {tuple(y.shape)}")
    _need(w, "w", N * k, rows=N)
    _need(counts, "counts", K)
    _need(offsets, "offsets", K + 1)
    _need(perm, "perm", N * k)
    # then devices, dtypes and layout
    _cuda(x, "x", None, 2)
    dev = x.device
    if indirect:
        for i, (a_i, b_i) in enumerate(zip(A, B)):
            _cuda(a_i, f"A[{i}]", x.dtype, 2, device=dev)
            _cuda(b_i, f"B[{i}]", x.dtype, 2, device=dev)
    else:
        _cuda(A, "A", x.dtype, 3, device=dev)
        _cuda(B, "B", x.dtype, 3, device=dev)
    _cuda(ids, "ids", torch.int32, device=dev)
    _cuda(y, "y", None, 2, device=dev)
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"y must be float32 or bfloat16, got {y.dtype}")
    _sized(w, "w", N * k, torch.float32, dev)
    _sized(counts, "counts", K, torch.int32, dev)
    _sized(offsets, "offsets", K + 1, torch.int32, dev)
    _sized(perm, "perm", N * k, torch.int32, dev)
    e = _p(_err_word(err_word, dev))
    s = _stream(stream, dev)
    lib = load_library()
    if indirect:
        a_ptrs = (ctypes.c_void_p * K)(*[t.data_ptr() for t in A])
        b_ptrs = (ctypes.c_void_p * K)(*[t.data_ptr() for t in B])
        _check("molora_lora_apply", lib.molora_lora_apply_indirect(
            _p(x), _dtype_code(x), N, d_in, d_out, ctypes.cast(a_ptrs, ctypes.c_void_p),
            ctypes.cast(b_ptrs, ctypes.c_void_p), K, r, _p(ids), _p(w), k, _p(counts), _p(offsets), _p(perm),
            float(scale), _p(y), 1 if y.dtype == torch.bfloat16 else 0, e, PATHS[path], s))
        return y
    if y.dtype == torch.bfloat16:
        _check("molora_lora_apply", lib.molora_lora_apply_bf16y(
            _p(x), _dtype_code(x), N, d_in, d_out, _p(A), _p(B), K, r, _p(ids), _p(w), k, _p(counts), _p(offsets),
            _p(perm), float(scale), _p(y), e, PATHS[path], s))
        return y

    def call(ws_ptr, ws_bytes):
        return lib.molora_lora_apply_ex(
            _p(x), _dtype_code(x), N, d_in, d_out, _p(A), _p(B), K, r, _p(ids), _p(w), k, _p(counts), _p(offsets),
            _p(perm), float(scale), _p(y), ws_ptr, ws_bytes, e, PATHS[path], s)
    if path in ("auto", "stacked") or ws is not None:
        _check("molora_lora_apply", _workspace(ws, dev, call))
    else:
        _check("molora_lora_apply", call(None, None))
    return y


@_on_tensor_device
def molora_route_vocab_lora_apply(tok, starts, x, A, B, y, scale, adapter=None, counts=None, offsets=None,
                                  perm=None, err_word=None, stream=None):
    """The whole vocabulary-routed step in one call: routing, dispatch and the apply (k = 1).
    Returns (adapter, counts, offsets, perm); y (fp32 or bf16) is updated in place."""
    return _route_vocab_lora_apply(tok, starts, x, A, B, y, scale, adapter, counts, offsets, perm, err_word, stream,
                                   None)


@_on_tensor_device
def molora_route_vocab_lora_apply_ex(tok, starts, x, A, B, y, scale, flags, adapter=None, counts=None, offsets=None,
                                     perm=None, err_word=None, stream=None):
    """molora_route_vocab_lora_apply with flags (INPUTS_READY: as for molora_route_vocab_dispatch_ex)."""
    return _route_vocab_lora_apply(tok, starts, x, A, B, y, scale, adapter, counts, offsets, perm, err_word, stream,
                                   int(flags))


def _route_vocab_lora_apply(tok, starts, x, A, B, y, scale, adapter, counts, offsets, perm, err_word, stream, flags):
    N, K = tok.numel(), starts.numel() - 1
    if x.dim() != 2 or x.shape[0] != N:
        raise ValueError("x must be [N, d_in] with one row per token")
    d_in = x.shape[1]
    if A.dim() != 3 or B.dim() != 3 or A.shape[0] != K or A.shape[1] != d_in or tuple(B.shape[:2]) != (K, A.shape[2]):
        raise ValueError("A must be [K, d_in, r] and B [K, r, d_out], with K = len(starts) - 1")
    r, d_out = A.shape[2], B.shape[2]
    if y.dim() != 2 or tuple(y.shape) != (N, d_out):
        raise ValueError(f"y must be [N, d_out] = {(N, d_out)}, got {tuple(y.shape)}")
    for name, t, n in (("adapter", adapter, N), ("counts", counts, K), ("offsets", offsets, K + 1), ("perm", perm, N)):
        _need(t, name, n)
    _cuda(tok, "tok", torch.int32, 1)
    dev = tok.device
    _cuda(starts, "starts", torch.int32, 1, device=dev)
    _cuda(x, "x", None, 2, device=dev)
    _cuda(A, "A", x.dtype, 3, device=dev)
    _cuda(B, "B", x.dtype, 3, device=dev)
    _cuda(y, "y", None, 2, device=dev)
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"y must be float32 or bfloat16, got {y.dtype}")
    if adapter is None:
        adapter = torch.empty(N, dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty(K, dtype=torch.int32, device=dev)
    if offsets is None:
        offsets = torch.empty(K + 1, dtype=torch.int32, device=dev)
    if perm is None:
        perm = torch.empty(N, dtype=torch.int32, device=dev)
    _sized(adapter, "adapter", N, torch.int32, dev)
    _sized(counts, "counts", K, torch.int32, dev)
    _sized(offsets, "offsets", K + 1, torch.int32, dev)
    _sized(perm, "perm", N, torch.int32, dev)
    args = (_p(tok), N, _p(starts), K, _p(x), _dtype_code(x), d_in, d_out, _p(A), _p(B), r, float(scale), _p(y),
            1 if y.dtype == torch.bfloat16 else 0, _p(adapter), _p(counts), _p(offsets), _p(perm),
            _p(_err_word(err_word, dev)))
    if flags is None:
        _check("molora_route_vocab_lora_apply",
               load_library().molora_route_vocab_lora_apply(*args, _stream(stream, dev)))
    else:
        _check("molora_route_vocab_lora_apply_ex",
               load_library().molora_route_vocab_lora_apply_ex(*args, flags, _stream(stream, dev)))
    return adapter, counts, offsets, perm


@_on_tensor_device
def molora_router_lora_apply(x, W1, W2, A, B, k, y, scale, b1=None, b2=None, logits=None, ids=None, w=None,
                             want_logits=True, err_word=None, ws=None, use_ws=True, stream=None):
    """The learned router and the top-k apply with one pass over x: returns
    (logits fp32 [N,K] or None, ids int32 [N,k], w fp32 [N,k]); y (fp32 or bf16) is updated in
    place.  ``use_ws=False`` restricts it to the one-kernel family (no workspace); otherwise a
    workspace is used where the library prefers the stacked pair (``ws`` if given, else a
    fresh buffer)."""
    if x.dim() != 2 or W1.dim() != 2 or W2.dim() != 2:
        raise ValueError("x must be [N, d_in], W1 [d_in, 64] and W2 [64, K]")
    N, d_in = x.shape
    if tuple(W1.shape) != (d_in, ROUTER_HIDDEN) or W2.shape[0] != ROUTER_HIDDEN:
        raise ValueError("W1 must be [d_in, 64] and W2 [64, K]")
    K = W2.shape[1]
    if A.dim() != 3 or B.dim() != 3 or A.shape[0] != K or A.shape[1] != d_in or tuple(B.shape[:2]) != (K, A.shape[2]):
        raise ValueError("A must be [K, d_in, r] and B [K, r, d_out], with K = W2.shape[1]")
    r, d_out = A.shape[2], B.shape[2]
    if y.dim() != 2 or tuple(y.shape) != (N, d_out):
        raise ValueError(f"y must be [N, d_out] = {(N, d_out)}, got {tuple(y.shape)}")
    _need(logits, "logits", N * K, rows=N)
    _need(ids, "ids", N * k, rows=N)
    _need(w, "w", N * k, rows=N)
    _need(b1, "b1", ROUTER_HIDDEN)
    _need(b2, "b2", K)
    _cuda(x, "x", None, 2)
    dev = x.device
    _cuda(W1, "W1", x.dtype, 2, device=dev)
    _cuda(W2, "W2", x.dtype, 2, device=dev)
    _cuda(A, "A", x.dtype, 3, device=dev)
    _cuda(B, "B", x.dtype, 3, device=dev)
    _cuda(y, "y", None, 2, device=dev)
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"y must be float32 or bfloat16, got {y.dtype}")
    _sized(b1, "b1", ROUTER_HIDDEN, torch.float32, dev)
    _sized(b2, "b2", K, torch.float32, dev)
    if logits is None and want_logits:
        logits = torch.empty(N, K, dtype=torch.float32, device=dev)
    if ids is None:
        ids = torch.empty(N, k, dtype=torch.int32, device=dev)
    if w is None:
        w = torch.empty(N, k, dtype=torch.float32, device=dev)
    _sized(logits, "logits", N * K, torch.float32, dev)
    _sized(ids, "ids", N * k, torch.int32, dev)
    _sized(w, "w", N * k, torch.float32, dev)
    e = _p(_err_word(err_word, dev))
    s = _stream(stream, dev)
    lib = load_library()

    def call(ws_ptr, ws_bytes):
        return lib.molora_router_lora_apply(
            _p(x), _dtype_code(x), N, d_in, d_out, _p(W1), _p(b1), _p(W2), _p(b2), _p(A), _p(B), K, r, k,
            float(scale), _p(logits), _p(ids), _p(w), _p(y), 1 if y.dtype == torch.bfloat16 else 0, ws_ptr,
            ws_bytes, e, s)
    if use_ws:
        _check("molora_router_lora_apply", _workspace(ws, dev, call))
    else:
        _check("molora_router_lora_apply", call(None, None))
    return logits, ids, w


@_on_tensor_device
def molora_lora_apply_static_ws(x, A, B, ids, y, scale, w=None, err_word=None, stream=None):
    """The stacked apply for callers that cannot allocate device memory: the workspace is a
    fixed scratch buffer inside the library (STATIC_SCRATCH_BYTES; N*K*r up to 4M), shared by
    every call on the device -- calls that may overlap on the GPU must be serialised.  The
    first call on a device looks the buffer up; make it before capturing a CUDA graph.
    Same results as molora_lora_apply(..., path="stacked"); y (fp32) is updated in place."""
    if x.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [N, d_in], A [K, d_in, r] and B [K, r, d_out]")
    N, d_in = x.shape
    K, _, r = A.shape
    d_out = B.shape[2]
    if A.shape[1] != d_in or tuple(B.shape[:2]) != (K, r):
        raise ValueError("A must be [K, d_in, r] and B [K, r, d_out]")
    k = _slots(ids, N)
    if y.dim() != 2 or tuple(y.shape) != (N, d_out):
        raise ValueError(f"y must be [N, d_out] = {(N, d_out)}, got {tuple(y.shape)}")
    _need(w, "w", N * k, rows=N)
    _cuda(x, "x", None, 2)
    dev = x.device
    _cuda(A, "A", x.dtype, 3, device=dev)
    _cuda(B, "B", x.dtype, 3, device=dev)
    _cuda(ids, "ids", torch.int32, device=dev)
    _cuda(y, "y", torch.float32, 2, device=dev)
    _sized(w, "w", N * k, torch.float32, dev)
    _check("molora_lora_apply_static_ws", load_library().molora_lora_apply_static_ws(
        _p(x), _dtype_code(x), N, d_in, d_out, _p(A), _p(B), K, r, _p(ids), _p(w), k, float(scale), _p(y),
        _p(_err_word(err_word, dev)), _stream(stream, dev)))
    return y


@_on_tensor_device
def molora_lora_apply_masked_pass(x, A, B, adapter_of, a, y, scale, err_word=None, path="auto", stream=None):
    """One per-sequence pass: y[t] += [adapter_of[t] == a] * scale * (x[t] A_a) B_a for every t."""
    if x.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [N, d_in], A [K, d_in, r] and B [K, r, d_out]")
    N, d_in = x.shape
    K, _, r = A.shape
    d_out = B.shape[2]
    if A.shape[1] != d_in or tuple(B.shape[:2]) != (K, r):
        raise ValueError("A must be [K, d_in, r] and B [K, r, d_out]")
    if adapter_of.dim() != 1 or adapter_of.numel() != N:
        raise ValueError(f"adapter_of must be [N] with N = {N}, got {tuple(adapter_of.shape)}")
    if y.dim() != 2 or tuple(y.shape) != (N, d_out):
        raise ValueError(f"y must be [N, d_out] = {(N, d_out)}, got {tuple(y.shape)}")
    _cuda(x, "x", None, 2)
    dev = x.device
    _cuda(A, "A", x.dtype, 3, device=dev)
    _cuda(B, "B", x.dtype, 3, device=dev)
    _cuda(adapter_of, "adapter_of", torch.int32, 1, device=dev)
    _cuda(y, "y", torch.float32, 2, device=dev)
    _check("molora_lora_apply_masked_pass", load_library().molora_lora_apply_masked_pass(
        _p(x), _dtype_code(x), N, d_in, d_out, _p(A), _p(B), K, r, _p(adapter_of), int(a), float(scale), _p(y),
        _p(_err_word(err_word, dev)), PATHS[path], _stream(stream, dev)))
    return y


_TYPE_CODES = {torch.float32: F32, torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3}


def _array(t: Optional[torch.Tensor], name: str, shape, dtype, device, rows=None):
    """The device pointer of a tensor argument of this shape, dtype and device index (None for None).
    That the device is a GPU is checked by _on_gpu, last, so that a mis-sized argument is reported as
    such.  With `rows`, any shape of as many elements and that many rows (0: whatever the rows) will do, as
    molora_lora_apply takes its slots' and its dispatch's arrays.  (One quick test first: a call has up to 18 of these.)"""
    if t is None:
        return None
    if (type(t) in _TENSORS and t.dtype is dtype and t.shape == shape and t.get_device() == device and
            t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.shape != shape and (rows is None or t.numel() != math.prod(shape) or (rows and t.shape[:1] != (rows,))):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != device:
        where = "the CPU" if device < 0 else f"cuda:{device}"
        raise ValueError(f"{name} is on {t.device}, expected {where} (all tensors of a call share one device)")
    return t.data_ptr()


_TENSORS = (torch.Tensor, torch.nn.Parameter)


def _call(name: str, device, *args):
    """Calls the library with the device of that index current and raises on a status that is not OK."""
    fn = getattr(_lib or load_library(), name)
    if device == torch._C._cuda_getDevice():
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != OK:
        _check(name, status)


def _on_gpu(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _matrix(t, name: str, types):
    """Checks a 2-D tensor argument that gives a call its sizes, and returns its dtype's code."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if t.shape[1] < 1:
        raise ValueError(f"{name} must have at least one column")
    if t.dtype not in types:
        raise ValueError(f"{name} must be one of {', '.join(str(d) for d in types)}, got {t.dtype}")
    return _TYPE_CODES[t.dtype]


def _named(value: str, name: str, table) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {', '.join(table)}, got {value!r}")
    return table[value]


def _error_word(err_word, device):
    return None if err_word is None else _err_word(err_word, torch.device("cuda", device)).data_ptr()


_FLOATS = (torch.bfloat16, torch.float32)
_E4M3, _BF16, _BF16_E4M3 = (torch.float8_e4m3fn,), (torch.bfloat16,), (torch.bfloat16, torch.float8_e4m3fn)


def _raw_stream(stream, device) -> int:
    """The handle of the given stream, else of the device's current one (torch's own accessor for
    compiled callers: the public one makes a Stream object, 2 us of a 6 us call)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream(stream, torch.device("cuda", device)).value or 0


def _new(like, shape, dtype, stream):
    """An output or workspace that a call makes for kernels on `stream`: from that stream's memory, so
    that neither work before it on the current stream nor whoever gets its memory next can meet them."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def molora_rmsnorm(x, weight, eps=1e-6, residual=None, sum_out=None, out=None, out8=None, scale8=None, stream=None):
    """Root-mean-square norm of x [N, d] (+ residual) by rows: returns (sum_out, out, out8, scale8).
    ``out`` (x's dtype) is made if neither it nor out8 is given; ``sum_out`` (x + residual) is made
    if there is a residual; out8 (float8_e4m3fn, with scale8 float32 [N]) is written if given.
    sum_out and out may each be x or residual."""
    code = _matrix(x, "x", _FLOATS)
    N, d = x.shape
    dev, dt, shape = x.get_device(), x.dtype, x.shape
    px = _array(x, "x", shape, dt, dev)
    pg = _array(weight, "weight", (d,), dt, dev)
    pr = _array(residual, "residual", shape, dt, dev)
    if weight is None:
        raise ValueError("weight must be a tensor")
    if not (isinstance(eps, (int, float)) and 0.0 < eps < math.inf):
        raise ValueError(f"eps must be positive and finite, got {eps!r}")
    if (out8 is None) != (scale8 is None):
        raise ValueError("out8 and scale8 go together")
    if residual is None and sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if residual is not None and sum_out is None:
        sum_out = _new(x, shape, dt, stream)
    if out is None and out8 is None:
        out = _new(x, shape, dt, stream)
    ps, po = _array(sum_out, "sum_out", shape, dt, dev), _array(out, "out", shape, dt, dev)
    p8 = _array(out8, "out8", shape, torch.float8_e4m3fn, dev)
    pc = _array(scale8, "scale8", (N,), torch.float32, dev)
    if ps is not None and ps == po and N:
        raise ValueError("sum_out and out must be different tensors")
    _on_gpu(x, "x")
    _call("molora_rmsnorm", dev, px, code, N, d, pr, ps, pg, eps, po, p8, pc, _raw_stream(stream, dev))
    return sum_out, out, out8, scale8


def molora_gate_topk(logits, k, score="softmax", bias=None, groups=1, keep_groups=1, group_top=1, renormalise=True,
                     scale=1.0, ids=None, w=None, err_word=None, stream=None):
    """Expert-style gate over logits [N, K] (bfloat16 or float32, K up to MAX_EXPERTS): returns
    (ids int32 [N, k], w float32 [N, k]), the k largest of score + bias within the keep_groups best
    of `groups` groups (each ranked by the sum of its group_top largest), with the scores as
    weights.  A token with fewer than k experts left has id -1 and weight 0 in its last slots."""
    code = _matrix(logits, "logits", _FLOATS)
    N, K = logits.shape
    dev = logits.get_device()
    score = _named(score, "score", SCORES)
    if K > MAX_EXPERTS:
        raise ValueError(f"at most {MAX_EXPERTS} experts, got {K}")
    if not 1 <= groups <= MAX_GROUPS or K % groups:
        raise ValueError(f"groups must be 1 to {MAX_GROUPS} and divide {K}, got {groups}")
    if group_top not in (1, 2) or K // groups < group_top:
        raise ValueError(f"group_top must be 1 or 2 and at most the group's {K // groups}, got {group_top}")
    if not 1 <= keep_groups <= groups:
        raise ValueError(f"keep_groups must be 1 to {groups}, got {keep_groups}")
    if not 1 <= k <= min(MAX_GATE_K, keep_groups * (K // groups)):
        raise ValueError(f"k must be 1 to {min(MAX_GATE_K, keep_groups * (K // groups))}, got {k}")
    pl = _array(logits, "logits", logits.shape, logits.dtype, dev)
    pb = _array(bias, "bias", (K,), torch.float32, dev)
    if ids is None:
        ids = _new(logits, (N, k), torch.int32, stream)
    if w is None:
        w = _new(logits, (N, k), torch.float32, stream)
    pi, pw = _array(ids, "ids", (N, k), torch.int32, dev), _array(w, "w", (N, k), torch.float32, dev)
    _on_gpu(logits, "logits")
    _call(
        "molora_gate_topk", dev, pl, code, N, K, score, pb, groups, keep_groups, group_top, k, 1 if renormalise else 0, scale, pi, pw,
        _error_word(err_word, dev), _raw_stream(stream, dev))
    return ids, w


def _y(y, N, d_out, dtype, like, stream):
    if y is None:
        if dtype not in _FLOATS:
            raise ValueError(f"out_dtype must be torch.float32 or torch.bfloat16, got {dtype}")
        return _new(like, (N, d_out), dtype, stream)
    if not isinstance(y, torch.Tensor) or y.dtype not in _FLOATS:
        raise ValueError("y must be a float32 or bfloat16 tensor")
    return y


def molora_linear(x, W, y=None, x_scale=None, w_scale=None, bias=None, act="none", residual=None,
                  out_dtype=torch.float32, err_word=None, stream=None):
    """y = act(x W^T + bias) + residual for x [N, d_in] and W [d_out, d_in] in bfloat16, float32 or
    float8_e4m3fn (then with float32 scales x_scale [N] and w_scale [d_out]).  ``y``: the output
    (float32 or bfloat16, residual's dtype; residual itself is allowed), else made in ``out_dtype``."""
    code = _matrix(x, "x", (torch.bfloat16, torch.float32, torch.float8_e4m3fn))
    N, d_in = x.shape
    dev = x.get_device()
    if not isinstance(W, torch.Tensor) or W.dim() != 2 or W.shape[0] < 1:
        raise ValueError("W must be a 2-D tensor [d_out, d_in]")
    d_out = W.shape[0]
    act = _named(act, "act", ACTIVATIONS)
    fp8 = code == E4M3
    if fp8 != (x_scale is not None) or fp8 != (w_scale is not None):
        raise ValueError("x_scale and w_scale are needed with float8_e4m3fn, and with nothing else")
    px = _array(x, "x", x.shape, x.dtype, dev)
    pw = _array(W, "W", (d_out, d_in), x.dtype, dev)
    psx = _array(x_scale, "x_scale", (N,), torch.float32, dev)
    psw = _array(w_scale, "w_scale", (d_out,), torch.float32, dev)
    pb = _array(bias, "bias", (d_out,), torch.float32, dev)
    y = _y(y, N, d_out, out_dtype, x, stream)
    pres = _array(residual, "residual", (N, d_out), y.dtype, dev)
    py = _array(y, "y", (N, d_out), y.dtype, dev)
    _on_gpu(x, "x")
    _call(
        "molora_linear", dev, px, code, psx, N, d_in, pw, psw, d_out, pb, act, pres, py, 1 if y.dtype == torch.bfloat16 else 0,
        _error_word(err_word, dev), _raw_stream(stream, dev))
    return y


def _on_device_of_x(fn):
    """_on_tensor_device for a call whose first argument is a tensor that says where the others are."""
    @functools.wraps(fn)
    def call(x, *args, **kwargs):
        if isinstance(x, torch.Tensor) and x.is_cuda and x.get_device() != torch._C._cuda_getDevice():
            with torch.cuda.device(x.device):
                return fn(x, *args, **kwargs)
        return fn(x, *args, **kwargs)
    return call


@_on_device_of_x
def molora_norm_linear_lora_apply(x, norm_weight, eps, W, A, B, ids, y, scale, w=None, counts=None, offsets=None,
                                  perm=None, residual=None, sum_out=None, h=None, h8=None, scale8=None, w_scale=None,
                                  bias=None, err_word=None, ws=None, stream=None):
    """A whole adapted projection: molora_rmsnorm of x (+ residual) into h, y = h W^T + bias, then
    molora_lora_apply of h in place on y.  With float8_e4m3fn W [d_out, d_in] (and w_scale [d_out])
    the base product reads the norm's 8-bit output.  Returns (y, sum_out, h, h8, scale8); the
    buffers that are not given are made."""
    code = _matrix(x, "x", _FLOATS)
    N, d_in = x.shape
    dev, dt, shape, f32, i32 = x.get_device(), x.dtype, x.shape, torch.float32, torch.int32
    if not isinstance(W, torch.Tensor) or W.dim() != 2 or W.shape[0] < 1 or W.dtype not in (dt, torch.float8_e4m3fn):
        raise ValueError("W must be [d_out, d_in] of x's dtype or float8_e4m3fn")
    d_out = W.shape[0]
    fp8 = W.dtype == torch.float8_e4m3fn
    if not isinstance(A, torch.Tensor) or not isinstance(B, torch.Tensor) or A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [K, d_in, r] and B [K, r, d_out]")
    K, r = A.shape[0], A.shape[2]
    k = _slots(ids, N)
    if fp8 != (w_scale is not None) or (not fp8 and (h8 is not None or scale8 is not None)):
        raise ValueError("w_scale is needed, and h8 and scale8 are taken, with float8_e4m3fn W only")
    if norm_weight is None:
        raise ValueError("norm_weight must be a tensor")
    if not (isinstance(eps, (int, float)) and 0.0 < eps < math.inf):
        raise ValueError(f"eps must be positive and finite, got {eps!r}")
    if residual is None and sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if not isinstance(y, torch.Tensor) or y.dtype not in _FLOATS:
        raise ValueError("y must be a float32 or bfloat16 tensor")
    px = _array(x, "x", x.shape, dt, dev)
    if residual is not None and sum_out is None:
        sum_out = _new(x, shape, dt, stream)
    if h is None:
        h = _new(x, shape, dt, stream)
    if fp8 and h8 is None:
        h8 = _new(x, shape, torch.float8_e4m3fn, stream)
    if fp8 and scale8 is None:
        scale8 = _new(x, (N,), f32, stream)
    if sum_out is not None and N and h.data_ptr() == sum_out.data_ptr():
        raise ValueError("h and sum_out must be different tensors")
    args = (px, code, N, d_in, _array(residual, "residual", x.shape, dt, dev), _array(sum_out, "sum_out", x.shape, dt, dev),
            _array(norm_weight, "norm_weight", (d_in,), dt, dev), eps, _array(h, "h", x.shape, dt, dev),
            _array(h8, "h8", x.shape, torch.float8_e4m3fn, dev), _array(scale8, "scale8", (N,), f32, dev),
            _array(W, "W", (d_out, d_in), W.dtype, dev), _TYPE_CODES[W.dtype], _array(w_scale, "w_scale", (d_out,), f32, dev),
            d_out, _array(bias, "bias", (d_out,), f32, dev), _array(A, "A", (K, d_in, r), dt, dev),
            _array(B, "B", (K, r, d_out), dt, dev), K, r, _array(ids, "ids", ids.shape, i32, dev),
            _array(w, "w", ids.shape, f32, dev, N), k, _array(counts, "counts", (K,), i32, dev, 0),
            _array(offsets, "offsets", (K + 1,), i32, dev, 0), _array(perm, "perm", (N * k,), i32, dev, 0), scale,
            _array(y, "y", (N, d_out), y.dtype, dev), 1 if y.dtype == torch.bfloat16 else 0)
    _on_gpu(x, "x")
    tail = (_error_word(err_word, dev), _raw_stream(stream, dev))
    lib = load_library()

    def call(ws_ptr, ws_bytes):
        return lib.molora_norm_linear_lora_apply(*args, ws_ptr, ws_bytes, *tail)
    if ws is not None or y.dtype != torch.bfloat16 or N > 256:
        _check("molora_norm_linear_lora_apply", _workspace(ws, x.device, call, stream))
    else:
        # no path needs a workspace (they are for fp32 y, or for many tokens' update), so none is asked for
        _check("molora_norm_linear_lora_apply", call(None, None))
    return y, sum_out, h, h8, scale8


def _scale_blocks(n):
    return -(-n // SCALE_BLOCK)


def _rows(x, types):
    """x, the 2-D tensor argument that gives a call its sizes: its data pointer, dtype's code, sizes and device index."""
    if type(x) not in _TENSORS or x.dtype not in types or x.dim() != 2 or not x.is_contiguous():
        code = _matrix(x, "x", types)
        return _array(x, "x", x.shape, x.dtype, x.get_device()), code, *x.shape, x.get_device()
    N, d = x.shape
    if d < 1:
        raise ValueError("x must have at least one column")
    return x.data_ptr(), _TYPE_CODES[x.dtype], N, d, x.get_device()


def molora_quantise_blocks(x, out8=None, scale8=None, stream=None):
    """x [N, d] (bfloat16 or float32) in float8_e4m3fn with a scale for each row's block of SCALE_BLOCK columns: returns
    (out8 [N, d], scale8 float32 [N, ceil(d / SCALE_BLOCK)]), made if not given."""
    px, code, N, d, dev = _rows(x, _FLOATS)
    shape, blocks = (N, d), (N, _scale_blocks(d))
    if out8 is None:
        out8 = _new(x, shape, torch.float8_e4m3fn, stream)
    if scale8 is None:
        scale8 = _new(x, blocks, torch.float32, stream)
    po, ps = _array(out8, "out8", shape, torch.float8_e4m3fn, dev), _array(scale8, "scale8", blocks, torch.float32, dev)
    _on_gpu(x, "x")
    _call("molora_quantise_blocks", dev, px, code, N, d, po, ps, _raw_stream(stream, dev))
    return out8, scale8


def molora_linear_blocks(x, x_scale, W, w_scale, y=None, bias=None, act="none", residual=None, out_dtype=torch.float32,
                         err_word=None, stream=None):
    """y = act(x W^T + bias) + residual for x [N, d_in] and W [d_out, d_in] in float8_e4m3fn with a scale for each block of
    SCALE_BLOCK: x_scale float32 [N, blocks of d_in] (molora_quantise_blocks), w_scale float32 [blocks of d_out, blocks of
    d_in].  d_in is a multiple of 16, x and W are 16-byte aligned.  y, bias, act, residual and out_dtype as for molora_linear."""
    px, _, N, d_in, dev = _rows(x, _E4M3)
    f32 = torch.float32
    if not isinstance(W, torch.Tensor) or W.dim() != 2 or W.shape[0] < 1:
        raise ValueError("W must be a 2-D tensor [d_out, d_in]")
    d_out, blocks = W.shape[0], _scale_blocks(d_in)
    act = _named(act, "act", ACTIVATIONS)
    if x_scale is None or w_scale is None:
        raise ValueError("x_scale and w_scale must be tensors")
    pw = _array(W, "W", (d_out, d_in), torch.float8_e4m3fn, dev)
    psx = _array(x_scale, "x_scale", (N, blocks), f32, dev)
    psw = _array(w_scale, "w_scale", (_scale_blocks(d_out), blocks), f32, dev)
    pb = _array(bias, "bias", (d_out,), f32, dev)
    y = _y(y, N, d_out, out_dtype, x, stream)
    pres = _array(residual, "residual", (N, d_out), y.dtype, dev)
    py = _array(y, "y", (N, d_out), y.dtype, dev)
    _on_gpu(x, "x")
    _call("molora_linear_blocks", dev, px, psx, N, d_in, pw, psw, d_out, pb, act, pres, py,
          1 if y.dtype == torch.bfloat16 else 0, _error_word(err_word, dev), _raw_stream(stream, dev))
    return y


def _gated_weights(W, d_in):
    """d_ff of W [2 d_ff, d_in]: the gate's rows before the up projection's."""
    if not isinstance(W, torch.Tensor) or W.dim() != 2 or W.shape[0] < 2 or W.shape[0] % 2:
        raise ValueError("W must be a 2-D tensor [2 * d_ff, d_in]")
    return W.shape[0] // 2


def molora_gated_linear(x, W, h=None, act="silu", x_scale=None, w_scale=None, err_word=None, stream=None):
    """The gated half of a feed-forward block: h = act(x Wg^T) * (x Wu^T), bfloat16 [N, d_ff], for x [N, d_in] and
    W = [Wg; Wu] [2 d_ff, d_in] in bfloat16 (d_in a multiple of 8), or in float8_e4m3fn (of 16) with a scale for each block of
    SCALE_BLOCK: x_scale float32 [N, blocks of d_in] and w_scale float32 [2 * blocks of d_ff, blocks of d_in].  x and W are
    16-byte aligned."""
    px, code, N, d_in, dev = _rows(x, _BF16_E4M3)
    bf16, f32 = torch.bfloat16, torch.float32
    d_ff, blocks = _gated_weights(W, d_in), _scale_blocks(d_in)
    act = _named(act, "act", ACTIVATIONS)
    fp8 = code == E4M3
    if fp8 != (x_scale is not None) or fp8 != (w_scale is not None):
        raise ValueError("x_scale and w_scale are needed with float8_e4m3fn, and with nothing else")
    pw = _array(W, "W", (2 * d_ff, d_in), x.dtype, dev)
    psx = _array(x_scale, "x_scale", (N, blocks), f32, dev)
    psw = _array(w_scale, "w_scale", (2 * _scale_blocks(d_ff), blocks), f32, dev)
    if h is None:
        h = _new(x, (N, d_ff), bf16, stream)
    ph = _array(h, "h", (N, d_ff), bf16, dev)
    _on_gpu(x, "x")
    _call("molora_gated_linear", dev, px, code, psx, N, d_in, pw, psw, d_ff, act, ph, _error_word(err_word, dev),
          _raw_stream(stream, dev))
    return h


def molora_gated_linear_backward(x, W, dh, act="silu", dx=None, dW=None, dproj=None, want_dx=True, want_dW=True,
                                 err_word=None, stream=None):
    """The gradients of molora_gated_linear's bfloat16 form from that of h, dh [N, d_ff]; the projections are made again.
    Returns (dx, dW, dproj): dx [N, d_in] and dW [2 d_ff, d_in], made if not given unless want_dx or want_dW is false
    (frozen weights need no dW), and dproj [N, 2, d_ff rounded up to 8], the projections' gradient (columns from d_ff on are
    unspecified), made if not given."""
    px, code, N, d_in, dev = _rows(x, _BF16)
    bf16 = torch.bfloat16
    d_ff = _gated_weights(W, d_in)
    act = _named(act, "act", ACTIVATIONS)
    if dh is None:
        raise ValueError("dh must be a tensor")
    pw = _array(W, "W", (2 * d_ff, d_in), bf16, dev)
    pdh = _array(dh, "dh", (N, d_ff), bf16, dev)
    if dx is None and want_dx:
        dx = _new(x, x.shape, bf16, stream)
    if dW is None and want_dW:
        dW = _new(x, W.shape, bf16, stream)
    proj = (N, 2, (d_ff + 7) // 8 * 8)
    if dproj is None:
        dproj = _new(x, proj, bf16, stream)
    pdx, pdw = _array(dx, "dx", x.shape, bf16, dev), _array(dW, "dW", W.shape, bf16, dev)
    pdp = _array(dproj, "dproj", proj, bf16, dev)
    _on_gpu(x, "x")
    _call("molora_gated_linear_backward", dev, px, code, N, d_in, pw, d_ff, act, pdh, pdp, pdx, pdw,
          _error_word(err_word, dev), _raw_stream(stream, dev))
    return dx, dW, dproj


@_on_tensor_device
def molora_selftest_bounded_wait(err_word, limit_us=1000, stream=None):
    """Runs one CTA whose mbarrier wait can never complete; it must give up after limit_us and
    set DEV_WAIT_TIMEOUT in err_word (a device int32 tensor)."""
    _cuda(err_word, "err_word", torch.int32)
    dev = err_word.device
    _err_word(err_word, dev)
    _check("molora_selftest_bounded_wait", load_library().molora_selftest_bounded_wait(
        int(limit_us), _p(err_word), _stream(stream, dev)))
    return err_word


def molora_select_path(dtype: torch.dtype, N: int, d_in: int, d_out: int, K: int, r: int, k: int) -> str:
    """The kernel family molora_lora_apply picks for this shape when it may use a workspace
    ("scalar", "grouped", "dense" or "stacked")."""
    code = BF16 if dtype == torch.bfloat16 else F32
    return PATH_NAMES[load_library().molora_select_path(code, N, d_in, d_out, K, r, k)]
