"""ctypes binding of the operators in include/moonep_ffn.h (argument marshalling only):
products with bias, activation and residual, their gradients, and the combine with
dropout.  Same rules as ``_lib``: dense CUDA tensors, the current stream unless one is
given, an exception on a non-zero status, no fallback; tensors are on the current
device."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import _check, _keep, _stream, moonep_dims

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}
OUT_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
BF16 = torch.bfloat16


class moonep_linear_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "K", "N", "act", "out_f32")]


_device = _lib._raw_device or torch.cuda.current_device


def _ptr(t, dtype, numel, name, allow_none=False):
    if t is None and allow_none:
        return None
    if (type(t) is torch.Tensor and t.dtype is dtype and t.is_cuda and t.get_device() == _device()
            and t.is_contiguous() and (numel is None or t.numel() == numel)):
        return t.data_ptr()
    p = _lib._ptr(t, dtype, numel, name, allow_none)
    if t is not None and t.get_device() != _device():
        raise ValueError(f"{name} is on device {t.get_device()}, the current one is {_device()}")
    return p


_ready = False


def library() -> ctypes.CDLL:
    global _ready
    lib = _lib.library()
    if _ready:
        return lib
    P, D = ctypes.c_void_p, ctypes.POINTER(moonep_dims)
    I32, I64, F64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    N, L = ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(moonep_linear_dims)
    sig = {
        "moonep_linear": [L] + [P] * 8,
        "moonep_linear_dx": [L, P, P, P, P, P],
        "moonep_linear_dw": [L, P, P, P, I32, P, P],
        "moonep_act_backward_workspace_bytes": [I64, I32, N],
        "moonep_act_backward": [I64, I32, I32, P, P, P, P, I32, P, P],
        "moonep_grouped_gemm_act": [D, P, I32, P, P, P, P, P, P, P],
        "moonep_grouped_act_backward_workspace_bytes": [D, N],
        "moonep_grouped_act_backward": [D, P, I32, P, P, P, P, I32, P, P],
        "moonep_combine_dropout": [D, P, P, P, P, P, F64, P, P],
        "moonep_combine_dropout_backward": [D, P, P, P, P, P, P, F64, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    _ready = True
    return lib


def _act(act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return code


def _int32(value, name):
    """A size for an int32 argument, whose higher bits ctypes would drop without a word."""
    if not -(1 << 31) <= value < 1 << 31:
        raise ValueError(f"{name} is {value}, past 32 bits")
    return value


def linear_dims(T, K, N, act="none", out_dtype=torch.bfloat16) -> moonep_linear_dims:
    """x [T, K] times w [K, N]; act: "none", "relu", "gelu", "silu" or "swiglu" (whose output has
    N / 2 columns); out_dtype: that of moonep_linear's out, bfloat16 or float32."""
    if out_dtype not in OUT_DTYPES:
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    return moonep_linear_dims(_int32(T, "T"), _int32(K, "K"), _int32(N, "N"), _act(act), OUT_DTYPES[out_dtype])


_linear: dict = {}  # of linear dims already seen, by their fields


def _linear_sizes(ld):
    """(T*K, K*N, T*N, N, elements of out, its dtype), kept: the fields of a ctypes structure take
    longer to read than a small call may last."""
    key = bytes(ld)
    got = _linear.get(key)
    if got is None:
        T, K, N = ld.T, ld.K, ld.N
        cols = N // 2 if ld.act == ACTIVATIONS["swiglu"] else N
        got = _keep(_linear, key, (T * K, K * N, T * N, N, T * cols,
                                   torch.float32 if ld.out_f32 else BF16))
    return got


def moonep_linear(ld, x, w, out, status, bias=None, residual=None, z=None, stream=None):
    """out = residual + act(x w + bias); status: an int32 CUDA tensor of one element, zeroed once."""
    TK, KN, TN, N, TC, dtype = _linear_sizes(ld)
    _check(library().moonep_linear(
        ctypes.byref(ld), _ptr(x, BF16, TK, "x"), _ptr(w, BF16, KN, "w"),
        _ptr(bias, torch.float32, N, "bias", True), _ptr(residual, BF16, TC, "residual", True),
        _ptr(out, dtype, TC, "out"), _ptr(z, BF16, TN, "z", True),
        _ptr(status, torch.int32, 1, "status"), _stream(stream)), "moonep_linear")


def moonep_linear_dx(ld, d_z, w, d_x, status, stream=None):
    TK, KN, TN = _linear_sizes(ld)[:3]
    _check(library().moonep_linear_dx(
        ctypes.byref(ld), _ptr(d_z, BF16, TN, "d_z"), _ptr(w, BF16, KN, "w"),
        _ptr(d_x, BF16, TK, "d_x"), _ptr(status, torch.int32, 1, "status"), _stream(stream)),
        "moonep_linear_dx")


def moonep_linear_dw(ld, x, d_z, d_w, status, accumulate=False, stream=None):
    TK, KN, TN = _linear_sizes(ld)[:3]
    _check(library().moonep_linear_dw(
        ctypes.byref(ld), _ptr(x, BF16, TK, "x"), _ptr(d_z, BF16, TN, "d_z"),
        _ptr(d_w, torch.float32, KN, "d_w"), int(bool(accumulate)),
        _ptr(status, torch.int32, 1, "status"), _stream(stream)), "moonep_linear_dw")


_act_scratch: dict = {}  # scratch bytes of (rows, cols) already asked for


def moonep_act_backward_workspace_bytes(rows: int, cols: int) -> int:
    size = _act_scratch.get((rows, cols))
    if size is None:
        n = ctypes.c_size_t(0)
        _check(library().moonep_act_backward_workspace_bytes(rows, _int32(cols, "cols"), ctypes.byref(n)),
               "moonep_act_backward_workspace_bytes")
        size = _keep(_act_scratch, (rows, cols), n.value)
    return size


def _scratch(t, need):
    if isinstance(t, torch.Tensor) and t.numel() < need:
        raise ValueError(f"scratch has {t.numel()} bytes, expected at least {need}")
    return _ptr(t, torch.uint8, None, "scratch", need == 0)


def moonep_act_backward(z, d_out, d_z, act="none", d_bias=None, scratch=None, accumulate=False,
                        stream=None):
    """z, d_z [..., N]; d_out [..., N], or [..., N / 2] for swiglu; d_bias float32 [N] with scratch
    (uint8, moonep_act_backward_workspace_bytes).  For act "none" z is not read and may be None, and
    so may d_z if d_bias is given."""
    code = _act(act)
    if not isinstance(d_out, torch.Tensor) or d_out.dim() < 1 or d_out.shape[-1] == 0:
        raise ValueError("d_out must be a tensor of rows")
    rows = d_out.numel() // d_out.shape[-1]
    cols = d_out.shape[-1] * (2 if act == "swiglu" else 1)
    n = rows * cols
    need = moonep_act_backward_workspace_bytes(rows, cols) if d_bias is not None else 0
    _check(library().moonep_act_backward(
        rows, _int32(cols, "cols"), code, _ptr(z, BF16, n, "z", code == 0), _ptr(d_out, BF16, None, "d_out"),
        _ptr(d_z, BF16, n, "d_z", code == 0), _ptr(d_bias, torch.float32, cols, "d_bias", True),
        int(bool(accumulate)), _scratch(scratch, need), _stream(stream)), "moonep_act_backward")


_plans: dict = {}  # of plan dims already seen, by their fields


def _plan_sizes(d):
    """(workspace bytes, N, N*H, N*Hp, E*H*Hp, R*B*H*Hp, E*Hp, R*S*Hp), kept as _linear_sizes keeps its."""
    key = bytes(d)
    got = _plans.get(key)
    if got is None:
        hh = d.H * d.Hp
        got = _keep(_plans, key, (_lib.moonep_plan_workspace_bytes(d), d.N, d.N * d.H, d.N * d.Hp, d.E * hh,
                                  d.R * d.B * hh, d.E * d.Hp, d.R * d.S * d.Hp))
    return got


def moonep_grouped_gemm_act(d, plan_ws, recv, w_home, w_slot, y, act="none", bias=None, z=None,
                            stream=None):
    """moonep_grouped_gemm with bias float32 [E, Hp] and an activation; z [R, C, Hp] if given."""
    code = _act(act)
    need, _, NH, NP, home, slots, EP, _ = _plan_sizes(d)
    _check(library().moonep_grouped_gemm_act(
        ctypes.byref(d), _ptr(plan_ws, torch.uint8, need, "plan_ws"), code, _ptr(recv, BF16, NH, "recv"),
        _ptr(w_home, BF16, home, "w_home"), _ptr(w_slot, BF16, slots, "w_slot", allow_none=slots == 0),
        _ptr(bias, torch.float32, EP, "bias", True),
        _ptr(y, BF16, NP // 2 if act == "swiglu" else NP, "y"), _ptr(z, BF16, NP, "z", True),
        _stream(stream)), "moonep_grouped_gemm_act")


_grouped_act: dict = {}  # scratch bytes of dims already asked for, by their fields


def moonep_grouped_act_backward_workspace_bytes(d: moonep_dims) -> int:
    key = bytes(d)
    size = _grouped_act.get(key)
    if size is None:
        n = ctypes.c_size_t(0)
        _check(library().moonep_grouped_act_backward_workspace_bytes(ctypes.byref(d),
                                                                     ctypes.byref(n)),
               "moonep_grouped_act_backward_workspace_bytes")
        size = _keep(_grouped_act, key, n.value)
    return size


def moonep_grouped_act_backward(d, plan_ws, z, d_y, d_z, act="none", d_bias=None, scratch=None,
                                accumulate=False, stream=None):
    """moonep_act_backward on the plan's rows; d_bias float32 [E, Hp] with scratch (uint8,
    moonep_grouped_act_backward_workspace_bytes)."""
    code = _act(act)
    need, _, _, n, _, _, EP, _ = _plan_sizes(d)
    sums = moonep_grouped_act_backward_workspace_bytes(d) if d_bias is not None else 0
    _check(library().moonep_grouped_act_backward(
        ctypes.byref(d), _ptr(plan_ws, torch.uint8, need, "plan_ws"), code,
        _ptr(z, BF16, n, "z", code == 0), _ptr(d_y, BF16, n // 2 if act == "swiglu" else n, "d_y"),
        _ptr(d_z, BF16, n, "d_z", code == 0), _ptr(d_bias, torch.float32, EP, "d_bias", True),
        int(bool(accumulate)), _scratch(scratch, sums), _stream(stream)), "moonep_grouped_act_backward")


def moonep_combine_dropout(d, plan_ws, y, gates, out, residual=None, p=0.0, rng=None, stream=None):
    """moonep_combine with dropout of probability p (rng: int64 CUDA tensor {seed, offset}), added to
    the residual."""
    need, N, _, NP, _, _, _, n = _plan_sizes(d)
    _check(library().moonep_combine_dropout(
        ctypes.byref(d), _ptr(plan_ws, torch.uint8, need, "plan_ws"), _ptr(y, BF16, NP, "y"),
        _ptr(gates, torch.float32, N, "gates"), _ptr(residual, BF16, n, "residual", True),
        _ptr(out, BF16, n, "out"), p, _ptr(rng, torch.int64, 2, "rng", True), _stream(stream)),
        "moonep_combine_dropout")


def moonep_combine_dropout_backward(d, plan_ws, y, gates, d_out, d_y, d_gates, p=0.0, rng=None,
                                    stream=None):
    """The gradient, with the p and rng of the forward pass."""
    need, N, _, NP, _, _, _, n = _plan_sizes(d)
    _check(library().moonep_combine_dropout_backward(
        ctypes.byref(d), _ptr(plan_ws, torch.uint8, need, "plan_ws"), _ptr(y, BF16, NP, "y"),
        _ptr(gates, torch.float32, N, "gates"), _ptr(d_out, BF16, n, "d_out"), _ptr(d_y, BF16, NP, "d_y"),
        _ptr(d_gates, torch.float32, N, "d_gates"), p, _ptr(rng, torch.int64, 2, "rng", True),
        _stream(stream)), "moonep_combine_dropout_backward")
