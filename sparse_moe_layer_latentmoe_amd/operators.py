"""The operators around the layer: routing from given logits and the norms
around a block, each with its gradient, and matrices in 8-bit floating point
(e4m3) with a scale for each block of 128, with their dense and grouped
products.

Thin wrappers over the C ABI (``include/lmoe.h``), like the rest of the
binding: they check tensors, allocate the outputs and marshal pointers; the
kernels do the work.  ``stream`` is a torch stream or a raw handle of the
tensors' device (None: that device's current stream); outputs and scratch are
allocated for that stream, and tensors of a device that is not the current
one are fine.  Nothing is recorded for autograd: the gradients are calls of
their own.
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


class LmoeFp8MatmulArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "x", "x_scales", "w", "w_scales", "rows", "offsets", "y")] + [
        (n, ctypes.c_int32) for n in ("y_type", "n_groups", "M", "x_rows", "N", "K")]


def declare(lib: ctypes.CDLL) -> None:
    """Declare the C signatures of this module's entry points."""
    P, I, L, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    R, A, G, M = (ctypes.POINTER(t) for t in (LmoeRouter, LmoeBlockNormArgs, LmoeBlockNormGrads,
                                              LmoeFp8MatmulArgs))
    for name, args, res in (
            ("lmoe_route_logits", [R, P, I, L, P, I, P, P, P], ctypes.c_int),
            ("lmoe_route_logits_backward", [R, P, I, L, P, P, I, P, P], ctypes.c_int),
            ("lmoe_block_norm", [A, P, P, P, P], ctypes.c_int),
            ("lmoe_block_norm_workspace_size", [A, G], Z),
            ("lmoe_block_norm_backward", [A, P, P, P, G, P, Z, P], ctypes.c_int),
            ("lmoe_quantize_fp8", [P, I, L, I, L, P, P, P], ctypes.c_int),
            ("lmoe_quantize_fp8_weight", [P, I, L, I, I, P, P, P], ctypes.c_int),
            ("lmoe_fp8_matmul_workspace_size", [M], Z),
            ("lmoe_fp8_matmul", [M, P, Z, P], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


def _check(t, what: str, dtypes, ndim=None, shape=None, device=None, dense: bool = True) -> None:
    """Raise unless ``t`` is a GPU tensor of one of ``dtypes`` and this shape,
    on GPU number ``device``; dense, or (not dense) with contiguous rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{what}: {t.dim()} dimensions, expected {ndim}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        if dense:
            raise ValueError(f"{what}: must be contiguous")
        if t.shape[-1] > 1 and t.stride(-1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
            raise ValueError(f"{what}: rows must be contiguous and not overlap")
    if t.get_device() != device:        # -1 where it is not a GPU tensor
        if not t.is_cuda:
            raise ValueError(f"{what}: must be a GPU tensor, got one on {t.device}")
        if device is not None:
            raise ValueError(f"{what}: on {t.device}, expected cuda:{device}")


def _no_graph(where: str, *tensors) -> None:
    """Raise where autograd would expect ``where`` to record a gradient
    (``_check`` speaks up for what is no tensor)."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and getattr(t, "requires_grad", False):
                raise ValueError(
                    f"{where}: an input requires a gradient, which this call does not record; "
                    f"call it from a torch.autograd.Function whose backward is {where}_backward, "
                    "or under torch.no_grad()")


def _type(t) -> int:
    return F32 if t is None else _TYPE[t.dtype]


def _row_stride(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


@contextlib.contextmanager
def _switched(device: int, stream):
    with torch.cuda.device(device):
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.current_stream() if stream is None else \
                torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream) or 0))
        if stream.device.index != device:
            raise ValueError(f"stream: on {stream.device}, the tensors are on cuda:{device}")
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


def _launch(device: int, stream):
    """Context with GPU ``device`` and ``stream`` current (so that allocations
    belong to that stream); yields the stream's handle."""
    if stream is None and device == torch._C._cuda_getDevice():
        return _OnCurrent(torch._C._cuda_getCurrentRawStream(device))
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
    that only orders the experts.  Logits that require a gradient are refused
    where autograd is recording (route_logits_backward computes it)."""
    _no_graph("route_logits", logits)
    _check(logits, "logits", _TYPE, ndim=2, dense=False)
    T, E = logits.shape
    if E != router.n_experts:
        raise ValueError(f"logits: {E} experts, the router has {router.n_experts}")
    if bias is not None:
        _check(bias, "bias", (torch.float32,), shape=(E,), device=logits.get_device())
    K = max(int(router.top_k), 0)
    with _launch(logits.get_device(), stream) as s:
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
    _check(topk_idx, "topk_idx", (torch.int32,), shape=(T, K), device=logits.get_device())
    _check(dw, "dw", (torch.float32,), shape=(T, K), device=logits.get_device())
    with _launch(logits.get_device(), stream) as s:
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
    dev = h.get_device()
    if y is not None:
        _check(y, "y", _TYPE, shape=(T, D), device=dev, dense=False)
    for name, t in (("pre_weight", pre_weight), ("post_weight", post_weight),
                    ("res_scale", res_scale)):
        if t is not None:
            _check(t, name, _TYPE, shape=(D,), device=dev)
    kind = GATE_NONE
    if gate is not None:
        _check(gate, "gate", _TYPE, device=dev)
        shape = gate.shape
        if shape == (D,):
            kind = GATE_CHANNEL
        elif shape == (T, D):
            kind = GATE_FULL
        elif shape == (T, 1):
            kind = GATE_TOKEN
        else:
            raise ValueError(f"gate: shape {tuple(shape)}, expected ({D},), ({T}, 1) or ({T}, {D})")
    return LmoeBlockNormArgs(
        h.data_ptr(), _ptr(y), _row_stride(h), 0 if y is None else _row_stride(y),
        _ptr(pre_weight), _ptr(post_weight), _ptr(res_scale), _ptr(gate), kind, _TYPE[h.dtype],
        BF16 if y is None else _TYPE[y.dtype], _type(pre_weight), _type(post_weight),
        _type(res_scale), _type(gate), T, D, eps)


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
    has y's (bf16 without y).  stats (want_stats) is what the backward needs.
    Inputs that require a gradient are refused where autograd is recording
    (block_norm_backward computes it)."""
    _no_graph("block_norm", h, y, pre_weight, post_weight, gate, res_scale)
    a = _norm_args(h, y, pre_weight, post_weight, gate, res_scale, eps)
    T, D = h.shape
    with _launch(h.get_device(), stream) as s:
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
    gpu = h.get_device()
    _check(stats, "stats", (torch.float32,), shape=(T, 2), device=gpu)
    if dh_out is not None:
        _check(dh_out, "dh_out", (h.dtype,), shape=(T, D), device=gpu)
    if dx is not None:
        if pre_weight is None:
            raise ValueError("dx: the forward had no pre_weight, so no x")
        _check(dx, "dx", (_y_dtype(y),), shape=(T, D), device=gpu)
    lib = load_library()
    with _launch(gpu, stream) as s:
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


# ---- 8-bit floating point ----------------------------------------------------

_E4M3 = torch.float8_e4m3fn


def quantize_fp8(x, stream=None):
    """(codes float8_e4m3fn [T, K], scales fp32 [T, ceil(K / 128)]) of
    activations x [T, K] (fp32 or bf16, rows may be strided): each block of
    128 values of a row has its own scale."""
    _check(x, "x", _TYPE, ndim=2, dense=False)
    T, K = x.shape
    with _launch(x.get_device(), stream) as s:
        codes = torch.empty((T, K), dtype=_E4M3, device=x.device)
        scales = torch.empty((T, (K + 127) // 128), dtype=torch.float32, device=x.device)
        _done(load_library().lmoe_quantize_fp8(_ptr(x), _TYPE[x.dtype], T, K, _row_stride(x),
                                               _ptr(codes), _ptr(scales), s),
              "lmoe_quantize_fp8")
    return codes, scales


def quantize_fp8_weight(w, stream=None):
    """(codes float8_e4m3fn like w, scales fp32 [..., ceil(N / 128),
    ceil(K / 128)]) of weights w [..., N, K] (fp32 or bf16): each 128 x 128
    block of a matrix has its own scale."""
    _check(w, "w", _TYPE)
    if w.dim() < 2:
        raise ValueError(f"w: {w.dim()} dimensions, expected at least 2")
    N, K = w.shape[-2:]
    lead = tuple(w.shape[:-2])
    n = w.numel() // (N * K) if N and K else 0
    with _launch(w.get_device(), stream) as s:
        codes = torch.empty(w.shape, dtype=_E4M3, device=w.device)
        scales = torch.empty((*lead, (N + 127) // 128, (K + 127) // 128), dtype=torch.float32,
                             device=w.device)
        _done(load_library().lmoe_quantize_fp8_weight(_ptr(w), _TYPE[w.dtype], n, N, K,
                                                      _ptr(codes), _ptr(scales), s),
              "lmoe_quantize_fp8_weight")
    return codes, scales


def fp8_matmul(x, x_scales, w, w_scales, offsets=None, rows=None, out_dtype=torch.bfloat16,
               out=None, stream=None):
    """y [M, N] = x w^T of quantised matrices (quantize_fp8, quantize_fp8_weight).

    x [X, K], w [N, K]; K a multiple of 128, N of 16.  ``rows`` (int32 [M]):
    row m of y reads x's row rows[m] (else row m).  ``offsets`` (int32
    [G + 1], ascending) with w [G, N, K]: rows offsets[g] .. offsets[g + 1] - 1
    take matrix g; rows of no group are not written (pass ``out`` to keep what
    they hold).  out_dtype: bf16 or fp32."""
    e4m3, f32 = (_E4M3,), (torch.float32,)
    _check(x, "x", e4m3, ndim=2)
    dev, gpu = x.device, x.get_device()
    X, K = x.shape
    _check(w, "w", e4m3, ndim=2 if offsets is None else 3, device=gpu)
    N = w.shape[-2]
    if w.shape[-1] != K:
        raise ValueError(f"w: {w.shape[-1]} columns, x has {K}")
    kb = (K + 127) // 128
    _check(x_scales, "x_scales", f32, shape=(X, kb), device=gpu)
    _check(w_scales, "w_scales", f32, shape=(*w.shape[:-2], (N + 127) // 128, kb), device=gpu)
    i32 = (torch.int32,)
    if offsets is not None:
        if w.shape[0] < 1:
            raise ValueError("w: no groups")
        _check(offsets, "offsets", i32, shape=(w.shape[0] + 1,), device=gpu)
    M = X
    if rows is not None:
        _check(rows, "rows", i32, ndim=1, device=gpu)
        M = rows.shape[0]
    if out is not None:
        _check(out, "out", _TYPE, shape=(M, N), device=gpu)
    elif out_dtype not in _TYPE:
        raise TypeError(f"out_dtype: {out_dtype}, expected torch.bfloat16 or torch.float32")
    lib = load_library()
    with _launch(gpu, stream) as s:
        y = torch.empty((M, N), dtype=out_dtype, device=dev) if out is None else out
        a = LmoeFp8MatmulArgs(_ptr(x), _ptr(x_scales), _ptr(w), _ptr(w_scales), _ptr(rows),
                              _ptr(offsets), _ptr(y), _TYPE[y.dtype],
                              0 if offsets is None else w.shape[0], M, X, N, K)
        nbytes = int(lib.lmoe_fp8_matmul_workspace_size(a))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        _done(lib.lmoe_fp8_matmul(a, _ptr(ws), nbytes, s), "lmoe_fp8_matmul")
    return y
