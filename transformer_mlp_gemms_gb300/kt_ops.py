"""Binding of ``include/kt_ops.h``: layer norm and its gradients, 8-bit rows and the 8-bit
linear layer, the mixture-of-experts layer for a few tokens, a gated block and a linear layer
with their gradients, AdamW, and the linear layer in 8-bit floating point with its quantiser.

The functions carry the names of the C entry points and take torch tensors: sizes and row
pitches come from the tensors, which may be row slices of wider ones (any stride between
rows, consecutive elements within one).  A tensor that does not fit (its device, type, shape
or strides) raises ``KtError`` with ``KT_ERR_INVALID`` before anything is launched, as the
library's own refusals do.  Nothing is computed here, and outputs are the caller's tensors.
Work goes to torch's current stream of the tensors' device unless ``stream`` names another;
tensors that other streams still use are the caller's to order, as with any torch call.

The checks are compiled (``csrc/kt_ops_py.cpp``, built beside the library): in Python they would
take longer than a small call does on the GPU.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import kt_mlp
from .kt_mlp import KT_ACT_GEGLU, KT_ACT_NONE, KT_ERR_INVALID, KtError, _check

MODULE_PATH = os.path.join(kt_mlp.HERE, "_build", "_kt_ops.so")
_VP, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float

KT_LAYERNORM_MAX_D = 16384
KT_LINEAR_I8_DOT_ROWS = 16
KT_MOE_MAX_TOKENS, KT_MOE_MAX_EXPERTS, KT_MOE_MAX_TOP_K = 64, 256, 16
KT_F32, KT_ADAMW_BLOCK = 2, 256
KT_LINEAR_FP8_FEW = 32


class kt_moe_options(ctypes.Structure):
    _fields_ = [(n, _I64) for n in ("max_tokens", "D", "F", "experts", "top_k")] + \
               [(n, ctypes.c_int32) for n in ("act", "dtype", "bias", "normalize")]


class kt_moe_tensors(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("X", _VP), ("ldx", _I64)] + \
               [(n, _VP) for n in ("W_router", "W_up", "W_down", "b_up", "b_down", "R", "Y", "ids", "weights")]


class kt_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, _VP) for n in ("param", "grad", "m", "v", "m_scale", "v_scale", "copy")] + \
               [("n", _I64), ("weight_decay", ctypes.c_double)]


class kt_adamw_options(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("param_dtype", "grad_dtype", "copy_dtype", "state_bits")] + \
               [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps")] + \
               [("step", _I64), ("step_device", _VP), ("grad_scale", _VP)]


# every entry point declared in include/kt_ops.h, with its ctypes signature
SIGNATURES = {
    "kt_layernorm_forward": ([_I64, _I64, _I32, _VP, _I64, _VP, _VP, _F32, _VP, _I64, _VP, _VP, _VP], _I32),
    "kt_layernorm_backward": ([_I64, _I64, _I32, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _I64, _VP, _VP, _VP,
                               ctypes.c_size_t, _VP], _I32),
    "kt_layernorm_backward_workspace": ([_I64, _I64], ctypes.c_size_t),
    "kt_quantize_rows": ([_I64, _I64, _I32, _I32, _VP, _I64, _VP, _I64, _VP, _VP], _I32),
    "kt_linear_i8": ([_I64, _I64, _I64, _I32, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _I64, _VP], _I32),
    "kt_linear_i8_status": ([_VP], _I32),
    "kt_linear_i8_debug_stall": ([_I32, _I64], _I32),
    "kt_moe_plan": ([ctypes.POINTER(kt_moe_options), ctypes.POINTER(_VP)], _I32),
    "kt_moe_run": ([_VP, ctypes.POINTER(kt_moe_tensors), _VP], _I32),
    "kt_moe_status": ([_VP], _I32),
    "kt_moe_debug_stall": ([_VP, _I32, _I64], _I32),
    "kt_moe_destroy": ([_VP], _I32),
    "kt_glu_forward": ([_I64] * 3 + [_I32] * 2 + [_VP, _I64, _VP, _VP, _VP, _I64, _VP, _I64, _VP], _I32),
    "kt_glu_backward_workspace": ([_I64] * 3, ctypes.c_size_t),
    "kt_glu_backward": ([_I64] * 3 + [_I32] * 2 + [_VP, _I64] * 3 + [_VP, _VP, _I64, _VP, _VP, _VP, ctypes.c_size_t, _VP], _I32),
    "kt_linear_forward": ([_I64] * 3 + [_I32, _VP, _I64, _VP, _VP, _VP, _I64, _VP], _I32),
    "kt_linear_backward_workspace": ([_I64] * 3, ctypes.c_size_t),
    "kt_linear_backward": ([_I64] * 3 + [_I32] + [_VP, _I64] * 2 + [_VP, _VP, _I64, _VP, _VP, _VP, ctypes.c_size_t, _VP], _I32),
    "kt_adamw": ([_I64, ctypes.POINTER(kt_adamw_tensor), ctypes.POINTER(kt_adamw_options), _VP], _I32),
    "kt_quantize_fp8": ([_I64, _I64, _I32, _I32, _VP, _I64, _VP, _I64, _VP, _VP], _I32),
    "kt_linear_fp8": ([_I64, _I64, _I64, _I32, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _I64, _VP], _I32),
    "kt_matmul_status": ([_VP], _I32),
    "kt_matmul_debug_stall": ([_I32, _I64], _I32),
}

_lib = None
_ext = None


def load():
    """The shared library with this header's signatures set, and the module of the tensor calls
    (``OSError`` if they have not been built)."""
    global _lib, _ext
    if _lib is None:
        lib = kt_mlp.load()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        if not os.path.exists(MODULE_PATH):
            raise OSError(f"{MODULE_PATH} not found: build it with `python -m transformer_mlp_gemms_gb300.build`")
        spec = importlib.util.spec_from_file_location("_kt_ops", MODULE_PATH)
        _ext = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_ext)
        _lib = lib
    return _lib


def _calls():
    """The module of the tensor calls."""
    if _ext is None:
        load()
    return _ext


def _fail(result, where: str):
    """A tensor call's refusal: a text, or the library's status."""
    if isinstance(result, str):
        raise KtError(KT_ERR_INVALID, where, result)
    _check(result, where)


def kt_layernorm_forward(X, gamma, beta, eps, Y, mean=None, rstd=None, stream=None) -> None:
    """Y = layer norm of the rows of X; mean and rstd (fp32 [M]) receive the statistics if given."""
    r = (_ext or _calls()).layernorm_forward(X, gamma, beta, eps, Y, mean, rstd, stream)
    if r is not None:
        _fail(r, "kt_layernorm_forward")


def kt_layernorm_backward_workspace(M: int, D: int) -> int:
    """Bytes of workspace of kt_layernorm_backward (0 for sizes that it refuses)."""
    return load().kt_layernorm_backward_workspace(M, D)


def layernorm_backward_workspace(M: int, D: int, device="cuda"):
    """A workspace tensor for kt_layernorm_backward, to be kept from call to call on one stream."""
    return torch.empty(kt_layernorm_backward_workspace(M, D), dtype=torch.uint8, device=device)


def kt_layernorm_backward(dY, X, gamma, mean, rstd, dX, dgamma=None, dbeta=None, workspace=None, stream=None) -> None:
    """dX, and with dgamma and dbeta (fp32 [D]) their sums over the rows, which need ``workspace``
    (``layernorm_backward_workspace``)."""
    r = (_ext or _calls()).layernorm_backward(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, workspace, stream)
    if r is not None:
        _fail(r, "kt_layernorm_backward")


def kt_quantize_rows(X, Q, scale, act: int = KT_ACT_NONE, stream=None) -> None:
    """Q (int8 [M][K]) and scale (fp32 [M]) of act(X); X is [M][K], or [M][2K] for KT_ACT_GEGLU."""
    r = (_ext or _calls()).quantize_rows(X, Q, scale, act, stream)
    if r is not None:
        _fail(r, "kt_quantize_rows")


def kt_linear_i8(Q, scale_x, W, scale_w, bias, Y, stream=None) -> None:
    """Y[m][n] = scale_x[m] scale_w[n] sum_k Q[m][k] W[n][k] (+ bias[n])."""
    r = (_ext or _calls()).linear_i8(Q, scale_x, W, scale_w, bias, Y, stream)
    if r is not None:
        _fail(r, "kt_linear_i8")


def kt_linear_i8_status(stream=None) -> int:
    """Waits for the stream and returns the status code of the device's kt_linear_i8 calls (does not
    raise on KT_ERR_TIMEOUT)."""
    return load().kt_linear_i8_status(kt_mlp._stream(stream))


def kt_linear_i8_debug_stall(enable: bool, limit_us: int = 0) -> None:
    _check(load().kt_linear_i8_debug_stall(int(bool(enable)), limit_us), "kt_linear_i8_debug_stall")


def kt_moe_plan(options: kt_moe_options) -> int:
    out = _VP()
    _check(load().kt_moe_plan(ctypes.byref(options), ctypes.byref(out)), "kt_moe_plan")
    return out.value


def kt_moe_run(plan: int, tensors: kt_moe_tensors, stream=None) -> None:
    _check(load().kt_moe_run(plan, ctypes.byref(tensors), kt_mlp._stream(stream)), "kt_moe_run")


def kt_moe_status(plan: int) -> int:
    """Waits for the plan's device and returns the status code (does not raise on KT_ERR_TIMEOUT)."""
    return load().kt_moe_status(plan)


def kt_moe_debug_stall(plan: int, enable: bool, limit_us: int = 0) -> None:
    _check(load().kt_moe_debug_stall(plan, int(bool(enable)), limit_us), "kt_moe_debug_stall")


def kt_moe_destroy(plan: int) -> None:
    _check(load().kt_moe_destroy(plan), "kt_moe_destroy")


class MoePlan:
    """Owning handle of a mixture-of-experts layer for up to ``max_tokens`` tokens; destroyed with
    the object.  ``run`` takes W_router [E][D], W_up [E][F_up][D], W_down [E][D][F] (F_up = F, or
    2F for KT_ACT_GEGLU: value rows, then gate rows), b_up [E][F_up] and b_down [E][D] iff
    ``bias``, and an optional residual R [T][D]."""

    def __init__(self, max_tokens, D, F, experts, top_k, act, dtype, bias=False, normalize=True):
        self.max_tokens, self.D, self.F, self.experts, self.top_k = max_tokens, D, F, experts, top_k
        self.bias, self.rows = bool(bias), 2 * F if act == KT_ACT_GEGLU else F
        self.handle = None
        self.handle = kt_moe_plan(kt_moe_options(max_tokens, D, F, experts, top_k, act, dtype, int(bool(bias)),
                                                 int(bool(normalize))))
        self._sizes = (dtype, D, F, self.rows, experts, top_k)

    def run(self, X, W_router, W_up, W_down, Y, b_up=None, b_down=None, R=None, ids=None, weights=None, stream=None):
        r = (_ext or _calls()).moe_run(self.handle, self._sizes, X, W_router, W_up, W_down, Y, b_up, b_down, R, ids, weights,
                                       stream)
        if r is not None:
            _fail(r, "kt_moe_run")

    def status(self) -> int:
        return kt_moe_status(self.handle)

    def close(self):
        if getattr(self, "handle", None):
            kt_moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def kt_glu_forward(X, W, bias, H, P, act: int, stream=None) -> None:
    """H = value * act(gate) with [value | gate] = X W^T (+ bias), W [2F][D]; P [M][2F] receives value and
    gate if given (``kt_glu_backward`` wants them)."""
    r = (_ext or _calls()).glu_forward(X, W, bias, H, P, act, stream)
    if r is not None:
        _fail(r, "kt_glu_forward")


def kt_glu_backward_workspace(M: int, D: int, F: int) -> int:
    """Bytes of workspace of kt_glu_backward (0 for sizes that it refuses)."""
    return load().kt_glu_backward_workspace(M, D, F)


def glu_backward_workspace(M: int, D: int, F: int, device="cuda"):
    """A workspace tensor for kt_glu_backward, to be kept from call to call on one stream."""
    return torch.empty(kt_glu_backward_workspace(M, D, F), dtype=torch.uint8, device=device)


def kt_glu_backward(dH, P, X, W, dX, dW, db, act: int, workspace, stream=None) -> None:
    """dX [M][D], dW [2F][D] and db (fp32 [2F]) from dH and the P that kt_glu_forward kept; each of the
    three may be None."""
    r = (_ext or _calls()).glu_backward(dH, P, X, W, dX, dW, db, act, workspace, stream)
    if r is not None:
        _fail(r, "kt_glu_backward")


def kt_linear_forward(X, W, bias, Y, stream=None) -> None:
    """Y = X W^T (+ bias), W [N][K]."""
    r = (_ext or _calls()).linear_forward(X, W, bias, Y, stream)
    if r is not None:
        _fail(r, "kt_linear_forward")


def kt_linear_backward_workspace(M: int, N: int, K: int) -> int:
    """Bytes of workspace of kt_linear_backward (0 for sizes that it refuses)."""
    return load().kt_linear_backward_workspace(M, N, K)


def linear_backward_workspace(M: int, N: int, K: int, device="cuda"):
    """A workspace tensor for kt_linear_backward, to be kept from call to call on one stream."""
    return torch.empty(kt_linear_backward_workspace(M, N, K), dtype=torch.uint8, device=device)


def kt_linear_backward(dY, X, W, dX, dW, db, workspace, stream=None) -> None:
    """dX [M][K], dW [N][K] and db (fp32 [N]); each may be None."""
    r = (_ext or _calls()).linear_backward(dY, X, W, dX, dW, db, workspace, stream)
    if r is not None:
        _fail(r, "kt_linear_backward")


def kt_adamw(params, grads, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, m_scales=None,
             v_scales=None, copies=None, grad_scale=None, stream=None) -> None:
    """One AdamW step over lists of contiguous tensors, in place.  ``m`` and ``v`` are float32, or float8_e4m3fn
    with ``m_scales`` and ``v_scales`` (float32, one for each KT_ADAMW_BLOCK values; ``v`` then holds the second
    moment's root).  ``step``: a number from 1 on, or an int64 tensor on the device.  ``weight_decay``: a number,
    or one for each tensor.  ``copies``: 16-bit tensors that receive fp32 parameters' rounding."""
    r = (_ext or _calls()).adamw(params, grads, m, v, step, lr, beta1, beta2, eps, weight_decay, m_scales, v_scales, copies,
                                 grad_scale, stream)
    if r is not None:
        _fail(r, "kt_adamw")


def kt_quantize_fp8(X, Q, scale, act: int = KT_ACT_NONE, stream=None) -> None:
    """Q (float8_e4m3fn [M][K]) and scale (fp32 [M][ceil(K / 128)]) of act(X); X is [M][K], or [M][2K] for
    KT_ACT_GEGLU."""
    r = (_ext or _calls()).quantize_fp8(X, Q, scale, act, stream)
    if r is not None:
        _fail(r, "kt_quantize_fp8")


def kt_linear_fp8(Q, scale_x, W, scale_w, bias, Y, stream=None) -> None:
    """Y = (Q scale_x) (W scale_w)^T (+ bias), scales for runs of 128 columns and blocks of 128 x 128."""
    r = (_ext or _calls()).linear_fp8(Q, scale_x, W, scale_w, bias, Y, stream)
    if r is not None:
        _fail(r, "kt_linear_fp8")


def kt_matmul_status(stream=None) -> int:
    """Waits for the stream and returns the status code of the device's products (does not raise on
    KT_ERR_TIMEOUT)."""
    return load().kt_matmul_status(kt_mlp._stream(stream))


def kt_matmul_debug_stall(enable: bool, limit_us: int = 0) -> None:
    _check(load().kt_matmul_debug_stall(int(bool(enable)), limit_us), "kt_matmul_debug_stall")
