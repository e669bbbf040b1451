"""ctypes binding of the operators in include/moonep_ops.h (argument marshalling
only): the router with its balance loss and gradient, and MXFP4 quantisation,
dispatch and grouped product.  Same rules as ``_lib``: dense CUDA tensors, the
current stream unless one is given, an exception on a non-zero status, no
fallback."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import _check, _keep, _ptr, _stream, _ws, moonep_dims

SCORES = {"softmax": 0, "sigmoid": 1}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}


class moonep_router_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "E", "K", "segment", "score", "normalise",
                                               "dtype")] + [("scale", ctypes.c_float)]

    @property
    def G(self):
        n = self.segment or self.T
        return (self.T + n - 1) // n

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype else torch.float32


_ready = False


def library() -> ctypes.CDLL:
    global _ready
    lib = _lib.library()
    if _ready:
        return lib
    P, R, D = ctypes.c_void_p, ctypes.POINTER(moonep_router_dims), ctypes.POINTER(moonep_dims)
    I32, I64 = ctypes.c_int32, ctypes.c_int64
    sig = {
        "moonep_router_workspace_bytes": [R, ctypes.POINTER(ctypes.c_size_t)],
        "moonep_router_forward": [R] + [P] * 10,
        "moonep_router_backward": [R] + [P] * 9,
        "moonep_mxfp4_quantize": [I64, I32, P, P, P, P],
        "moonep_mxfp4_dequantize": [I64, I32, P, P, P, P],
        "moonep_mxfp4_quantize_weights": [I32, I32, I32, P, P, P, P],
        "moonep_mxfp4_prefetch_weights": [D, P, P, P, P, P, P],
        "moonep_mxfp4_dispatch": [D, P, P, P, P, P],
        "moonep_mxfp4_grouped_gemm": [D, P, P, P, P, P, P, P, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    _ready = True
    return lib


def router_dims(T, E, K, segment=0, score="softmax", normalise=True, scale=1.0,
                dtype=torch.float32) -> moonep_router_dims:
    """segment: tokens per segment of the balance loss (0: all T); score: "softmax" or
    "sigmoid"; dtype: that of the logits, float32 or bfloat16."""
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    if dtype not in DTYPES:
        raise ValueError(f"router logits must be float32 or bfloat16, got {dtype}")
    return moonep_router_dims(T, E, K, segment, SCORES[score], int(bool(normalise)), DTYPES[dtype],
                              scale)


_sizes: dict = {}  # of router dims already seen, by their fields


def _router_sizes(rd):
    """(workspace bytes, T*E, T*K, G*E, G, logits dtype), kept: the fields of a ctypes structure
    take longer to read than a small call may last."""
    lib, key = library(), bytes(rd)
    got = _sizes.get(key)
    if got is None:
        n = ctypes.c_size_t(0)
        _check(lib.moonep_router_workspace_bytes(ctypes.byref(rd), ctypes.byref(n)),
               "moonep_router_workspace_bytes")
        got = _keep(_sizes, key, (n.value, rd.T * rd.E, rd.T * rd.K, rd.G * rd.E, rd.G,
                                  rd.torch_dtype))
    return got


def moonep_router_workspace_bytes(rd: moonep_router_dims) -> int:
    return _router_sizes(rd)[0]


def moonep_router_forward(rd, logits, topk_idx, gates, token_mask=None, ws=None, counts=None,
                          prob_sum=None, seg_tokens=None, loss=None, stream=None):
    """The balance outputs (ws, counts, prob_sum, seg_tokens, loss) are all given or all None."""
    need, TE, TK, GE, G, dtype = _router_sizes(rd)
    if ws is not None and isinstance(ws, torch.Tensor) and ws.numel() < need:
        raise ValueError(f"ws has {ws.numel()} bytes, expected at least {need}")
    _check(library().moonep_router_forward(
        ctypes.byref(rd), _ptr(logits, dtype, TE, "logits"),
        _ptr(token_mask, torch.uint8, rd.T, "token_mask", True) if token_mask is not None else None,
        _ptr(topk_idx, torch.int32, TK, "topk_idx"), _ptr(gates, torch.float32, TK, "gates"),
        _ptr(ws, torch.uint8, None, "ws", True), _ptr(counts, torch.int32, GE, "counts", True),
        _ptr(prob_sum, torch.float32, GE, "prob_sum", True),
        _ptr(seg_tokens, torch.int32, G, "seg_tokens", True),
        _ptr(loss, torch.float32, 1, "loss", True), _stream(stream)), "moonep_router_forward")


def moonep_router_backward(rd, logits, topk_idx, d_logits, d_gates=None, token_mask=None,
                           counts=None, seg_tokens=None, d_loss=None, stream=None):
    """counts, seg_tokens and d_loss are all given or all None; d_gates may be None with them."""
    _, TE, TK, GE, G, dtype = _router_sizes(rd)
    _check(library().moonep_router_backward(
        ctypes.byref(rd), _ptr(logits, dtype, TE, "logits"),
        _ptr(token_mask, torch.uint8, rd.T, "token_mask", True) if token_mask is not None else None,
        _ptr(topk_idx, torch.int32, TK, "topk_idx"),
        _ptr(d_gates, torch.float32, TK, "d_gates", True),
        _ptr(counts, torch.int32, GE, "counts", True),
        _ptr(seg_tokens, torch.int32, G, "seg_tokens", True),
        _ptr(d_loss, torch.float32, 1, "d_loss", True),
        _ptr(d_logits, dtype, TE, "d_logits"), _stream(stream)), "moonep_router_backward")


def mxfp4_scale_pitch(cols: int) -> int:
    """Bytes of a row of scales: cols / 32, padded to a multiple of 16."""
    return (cols // 32 + 15) // 16 * 16


def _rows(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() < 1 or t.shape[-1] == 0:
        raise ValueError(f"{name} must be a tensor of rows")
    return t.numel() // t.shape[-1]


def moonep_mxfp4_quantize(src, codes, scales, stream=None):
    """src bf16 [..., cols] to codes uint8 [..., cols/2] and scales uint8 [..., pitch]."""
    rows, cols = _rows(src, "src"), src.shape[-1]
    _check(library().moonep_mxfp4_quantize(
        rows, cols, _ptr(src, torch.bfloat16, None, "src"),
        _ptr(codes, torch.uint8, rows * cols // 2, "codes"),
        _ptr(scales, torch.uint8, rows * mxfp4_scale_pitch(cols), "scales"), _stream(stream)),
        "moonep_mxfp4_quantize")


def moonep_mxfp4_dequantize(codes, scales, dst, stream=None):
    """codes and scales of moonep_mxfp4_quantize (or _quantize_weights) to dst bf16 [..., cols]."""
    rows, cols = _rows(dst, "dst"), dst.shape[-1]
    _check(library().moonep_mxfp4_dequantize(
        rows, cols, _ptr(codes, torch.uint8, rows * cols // 2, "codes"),
        _ptr(scales, torch.uint8, rows * mxfp4_scale_pitch(cols), "scales"),
        _ptr(dst, torch.bfloat16, None, "dst"), _stream(stream)), "moonep_mxfp4_dequantize")


def moonep_mxfp4_quantize_weights(w, codes, scales, stream=None):
    """w bf16 [n, H, Hp] to codes uint8 [n, Hp, H/2] and scales uint8 [n, Hp, pitch(H)]."""
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be a tensor [n, H, Hp]")
    n, H, Hp = w.shape
    _check(library().moonep_mxfp4_quantize_weights(
        n, H, Hp, _ptr(w, torch.bfloat16, None, "w"),
        _ptr(codes, torch.uint8, n * Hp * (H // 2), "codes"),
        _ptr(scales, torch.uint8, n * Hp * mxfp4_scale_pitch(H), "scales"), _stream(stream)),
        "moonep_mxfp4_quantize_weights")


def _weights(d, codes, scales, n, name, allow_none=False):
    return (_ptr(codes, torch.uint8, n * d.Hp * (d.H // 2), f"{name}_codes", allow_none),
            _ptr(scales, torch.uint8, n * d.Hp * mxfp4_scale_pitch(d.H), f"{name}_scales",
                 allow_none))


def moonep_mxfp4_prefetch_weights(d, plan_ws, home_codes, home_scales, slot_codes, slot_scales,
                                  stream=None):
    _check(library().moonep_mxfp4_prefetch_weights(
        ctypes.byref(d), _ws(d, plan_ws), *_weights(d, home_codes, home_scales, d.E, "home"),
        *_weights(d, slot_codes, slot_scales, d.R * d.B, "slot", d.B == 0), _stream(stream)),
        "moonep_mxfp4_prefetch_weights")


def moonep_mxfp4_dispatch(d, plan_ws, x, recv_codes, recv_scales, stream=None):
    _check(library().moonep_mxfp4_dispatch(
        ctypes.byref(d), _ws(d, plan_ws), _ptr(x, torch.bfloat16, d.R * d.S * d.H, "x"),
        _ptr(recv_codes, torch.uint8, d.N * (d.H // 2), "recv_codes"),
        _ptr(recv_scales, torch.uint8, d.N * mxfp4_scale_pitch(d.H), "recv_scales"),
        _stream(stream)), "moonep_mxfp4_dispatch")


def moonep_mxfp4_grouped_gemm(d, plan_ws, recv_codes, recv_scales, home_codes, home_scales,
                              slot_codes, slot_scales, y, stream=None):
    _check(library().moonep_mxfp4_grouped_gemm(
        ctypes.byref(d), _ws(d, plan_ws),
        _ptr(recv_codes, torch.uint8, d.N * (d.H // 2), "recv_codes"),
        _ptr(recv_scales, torch.uint8, d.N * mxfp4_scale_pitch(d.H), "recv_scales"),
        *_weights(d, home_codes, home_scales, d.E, "home"),
        *_weights(d, slot_codes, slot_scales, d.R * d.B, "slot", d.B == 0),
        _ptr(y, torch.bfloat16, d.N * d.Hp, "y"), _stream(stream)), "moonep_mxfp4_grouped_gemm")
