"""The operators around the layer: routing from given logits and the norms
around a block, each with its gradient.

Thin wrappers over the C ABI (``include/lmoe.h``), like the rest of the
binding: they check tensors, allocate the outputs and marshal pointers; the
kernels do the work.  ``stream`` is a torch stream or a raw handle of the
tensors' device (None: that device's current stream); outputs and scratch are
allocated for that stream, and tensors of a device that is not the current
one are fine.
"""

from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import LMOE_OK, LmoeError, _ptr, load_library

F32, BF16 = 0, 1                                    # lmoe_dtype
SCORE_SIGMOID, SCORE_SOFTMAX = 0, 1                 # lmoe_score
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3   # lmoe_gate

_TYPE = {torch.float32: F32, torch.bfloat16: BF16}


class LmoeRouter(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_experts", "top_k", "score", "n_group", "topk_group", "group_score",
        "renormalise")] + [("scale", ctypes.c_float)]


class LmoeBlockNormArgs(ctypes.Structure):
    _fields_ = [
        ("h", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("h_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
        ("pre_weight", ctypes.c_void_p), ("post_weight", ctypes.c_void_p),
        ("res_scale", ctypes.c_void_p), ("gate", ctypes.c_void_p),
        ("gate_kind", ctypes.c_int32), ("h_type", ctypes.c_int32), ("y_type", ctypes.c_int32),
        ("pre_type", ctypes.c_int32), ("post_type", ctypes.c_int32),
        ("res_scale_type", ctypes.c_int32), ("gate_type", ctypes.c_int32),
        ("T", ctypes.c_int32), ("D", ctypes.c_int32), ("eps", ctypes.c_float)]


class LmoeBlockNormGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "dh", "dy", "dpre_weight", "dpost_weight", "dres_scale", "dgate")]


def declare(lib: ctypes.CDLL) -> None:
    """Declare the C signatures of this module's entry points."""
    P, I, L, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    R, A, G = (ctypes.POINTER(t) for t in (LmoeRouter, LmoeBlockNormArgs, LmoeBlockNormGrads))
    for name, args, res in (
            ("lmoe_route_logits", [R, P, I, L, P, I, P, P, P], ctypes.c_int),
            ("lmoe_route_logits_backward", [R, P, I, L, P, P, I, P, P], ctypes.c_int),
            ("lmoe_block_norm", [A, P, P, P, P], ctypes.c_int),
            ("lmoe_block_norm_workspace_size", [A, G], Z),
            ("lmoe_block_norm_backward", [A, P, P, P, G, P, Z, P], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


def _check(t, what: str, dtypes, ndim=None, shape=None, device=None, dense: bool = True) -> None:
    """Raise unless ``t`` is a GPU tensor of one of ``dtypes`` and this shape;
    dense, or (not dense) with its last axis contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{what}: {t.dim()} dimensions, expected {ndim}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dense:
        if not t.is_contiguous():
            raise ValueError(f"{what}: must be contiguous")
    elif t.shape[-1] > 1 and t.stride(-1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what}: rows must be contiguous and not overlap")
    if t.device.type != "cuda":
        raise ValueError(f"{what}: must be a GPU tensor, got one on {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")


def _row_stride(t) -> int:
    return int(t.stride(0)) if t.shape[0] > 1 else int(t.shape[1])


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device):
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.current_stream() if stream is None else \
                torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream) or 0))
        if stream.device != device:
            raise ValueError(f"stream: on {stream.device}, the tensors are on {device}")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


class _OnCurrent:
    """The launch context of the usual case: the tensors' device is current
    and its current stream is meant."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *a):
        return False


def _launch(device, stream):
    """Context with ``device`` and ``stream`` current (so that allocations
    belong to that stream); yields the stream's handle."""
    if stream is None and device.index == torch.cuda.current_device():
        return _OnCurrent(torch.cuda.current_stream().cuda_stream)
    return _switched(device, stream)


def _done(st: int, where: str) -> None:
    if st != LMOE_OK:
        raise LmoeError(st, where)


# ---- routing ---------------------------------------------------------------


def make_router(n_experts: int, top_k: int, score: int = SCORE_SIGMOID, n_group: int = 1,
                topk_group: int = 1, group_score: int = 2, renormalise: bool = True,
                scale: float = 1.0) -> LmoeRouter:
    """How logits become experts and weights (lmoe_router of lmoe.h): sigmoid
    or softmax scores, ``topk_group`` of ``n_group`` groups by the sum of
    their ``group_score`` best scores, ``top_k`` experts, weights that sum to
    ``scale`` (renormalise) or are ``scale`` times the scores."""
    return LmoeRouter(int(n_experts), int(top_k), int(score), int(n_group), int(topk_group),
                      int(group_score), int(bool(renormalise)), float(scale))


def route_logits(router: LmoeRouter, logits, bias=None, stream=None):
    """(topk_idx int32 [T, K], ascending ids; topk_w fp32 [T, K]) from logits
    [T, E] (fp32 or bf16; rows may be strided) and an optional fp32 [E] bias
    that only orders the experts."""
    _check(logits, "logits", _TYPE, ndim=2, dense=False)
    T, E = logits.shape
    if E != router.n_experts:
        raise ValueError(f"logits: {E} experts, the router has {router.n_experts}")
    if bias is not None:
        _check(bias, "bias", (torch.float32,), shape=(E,), device=logits.device)
    K = max(int(router.top_k), 0)
    with _launch(logits.device, stream) as s:
        idx = torch.empty((T, K), dtype=torch.int32, device=logits.device)
        w = torch.empty((T, K), dtype=torch.float32, device=logits.device)
        _done(load_library().lmoe_route_logits(
            router, _ptr(logits), _TYPE[logits.dtype], _row_stride(logits), _ptr(bias), T,
            _ptr(idx), _ptr(w), s), "lmoe_route_logits")
    return idx, w


def route_logits_backward(router: LmoeRouter, logits, topk_idx, dw, stream=None):
    """The gradient of ``topk_w`` in the logits (dense, the logits' dtype)
    from ``dw`` fp32 [T, K], the selection held fixed."""
    _check(logits, "logits", _TYPE, ndim=2, dense=False)
    T, E = logits.shape
    if E != router.n_experts:
        raise ValueError(f"logits: {E} experts, the router has {router.n_experts}")
    K = int(router.top_k)
    _check(topk_idx, "topk_idx", (torch.int32,), shape=(T, K), device=logits.device)
    _check(dw, "dw", (torch.float32,), shape=(T, K), device=logits.device)
    with _launch(logits.device, stream) as s:
        dl = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
        _done(load_library().lmoe_route_logits_backward(
            router, _ptr(logits), _TYPE[logits.dtype], _row_stride(logits), _ptr(topk_idx),
            _ptr(dw), T, _ptr(dl), s), "lmoe_route_logits_backward")
    return dl


# ---- the norms around a block ----------------------------------------------


@dataclass
class BlockNormGrads:
    """Gradients of one block_norm call; None where the input was absent."""
    dh: object = None
    dy: object = None
    dpre_weight: object = None
    dpost_weight: object = None
    dres_scale: object = None
    dgate: object = None


def _norm_args(h, y, pre_weight, post_weight, gate, res_scale, eps) -> LmoeBlockNormArgs:
    _check(h, "h", _TYPE, ndim=2, dense=False)
    T, D = h.shape
    dev = h.device
    if y is not None:
        _check(y, "y", _TYPE, shape=(T, D), device=dev, dense=False)
    a = LmoeBlockNormArgs()
    for name, t in (("pre", pre_weight), ("post", post_weight), ("res_scale", res_scale)):
        if t is not None:
            _check(t, name if name == "res_scale" else name + "_weight", _TYPE, shape=(D,),
                   device=dev)
            setattr(a, name if name == "res_scale" else name + "_weight", t.data_ptr())
            setattr(a, name + "_type", _TYPE[t.dtype])
    if gate is not None:
        shape = tuple(gate.shape) if isinstance(gate, torch.Tensor) else None
        kind = {(D,): GATE_CHANNEL, (T, D): GATE_FULL}.get(shape)
        if shape == (T, 1) and D != 1:
            kind = GATE_TOKEN
        if shape is not None and kind is None:
            raise ValueError(f"gate: shape {shape}, expected ({D},), ({T}, 1) or ({T}, {D})")
        _check(gate, "gate", _TYPE, device=dev)
        a.gate, a.gate_kind, a.gate_type = gate.data_ptr(), kind, _TYPE[gate.dtype]
    a.h, a.h_stride, a.h_type = h.data_ptr(), _row_stride(h), _TYPE[h.dtype]
    if y is not None:
        a.y, a.y_stride, a.y_type = y.data_ptr(), _row_stride(y), _TYPE[y.dtype]
    else:
        a.y_type = BF16
    a.T, a.D, a.eps = T, D, eps
    return a


def _y_dtype(y):
    return torch.bfloat16 if y is None else y.dtype


def block_norm(h, y=None, pre_weight=None, post_weight=None, gate=None, res_scale=None,
               eps: float = 1e-5, want_stats: bool = False, stream=None):
    """(h_out, x, stats): h_out = res_scale h + gate n with n = RMSNorm(y) *
    post_weight (n = y without post_weight) and x = RMSNorm(h_out) *
    pre_weight (None without pre_weight).

    h: residual stream [T, D]; y: the block's output [T, D] (None: 0); each
    fp32 or bf16, rows may be strided.  pre_weight, post_weight, res_scale:
    [D] or None.  gate: [D], [T, 1], [T, D] or None.  h_out has h's dtype, x
    has y's (bf16 without y).  stats (want_stats) is what the backward needs."""
    a = _norm_args(h, y, pre_weight, post_weight, gate, res_scale, eps)
    T, D = h.shape
    with _launch(h.device, stream) as s:
        h_out = torch.empty((T, D), dtype=h.dtype, device=h.device)
        x = torch.empty((T, D), dtype=_y_dtype(y), device=h.device) \
            if pre_weight is not None else None
        stats = torch.empty((T, 2), dtype=torch.float32, device=h.device) if want_stats else None
        _done(load_library().lmoe_block_norm(a, _ptr(h_out), _ptr(x), _ptr(stats), s),
              "lmoe_block_norm")
    return h_out, x, stats


def block_norm_backward(h, y, stats, dh_out=None, dx=None, pre_weight=None, post_weight=None,
                        gate=None, res_scale=None, eps: float = 1e-5,
                        stream=None) -> BlockNormGrads:
    """Gradients of block_norm's inputs (each in its input's dtype) from the
    gradients of h_out (h's dtype) and x (y's dtype); None counts as 0.  The
    other arguments are the forward's; stats is what it returned."""
    a = _norm_args(h, y, pre_weight, post_weight, gate, res_scale, eps)
    T, D = h.shape
    dev = h.device
    _check(stats, "stats", (torch.float32,), shape=(T, 2), device=dev)
    if dh_out is not None:
        _check(dh_out, "dh_out", (h.dtype,), shape=(T, D), device=dev)
    if dx is not None:
        if pre_weight is None:
            raise ValueError("dx: the forward had no pre_weight, so no x")
        _check(dx, "dx", (_y_dtype(y),), shape=(T, D), device=dev)
    lib = load_library()
    with _launch(dev, stream) as s:
        g = BlockNormGrads(dh=torch.empty((T, D), dtype=h.dtype, device=dev))
        if y is not None:
            g.dy = torch.empty((T, D), dtype=y.dtype, device=dev)
        for name, t in (("dpre_weight", pre_weight), ("dpost_weight", post_weight),
                        ("dres_scale", res_scale), ("dgate", gate)):
            if t is not None:
                setattr(g, name, torch.empty_like(t))
        out = LmoeBlockNormGrads(*[_ptr(getattr(g, n)) for n, _ in LmoeBlockNormGrads._fields_])
        nbytes = int(lib.lmoe_block_norm_workspace_size(a, out))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        _done(lib.lmoe_block_norm_backward(a, _ptr(stats), _ptr(dh_out), _ptr(dx), out, _ptr(ws),
                                           nbytes, s), "lmoe_block_norm_backward")
    return g
