"""Binding of ``include/kt_ops.h``: layer norm and its gradients, 8-bit rows and the 8-bit
linear layer, and the mixture-of-experts layer for a few tokens.

The functions carry the names of the C entry points and take torch tensors: sizes and row
pitches come from the tensors, which may be row slices of wider ones (any stride between
rows, consecutive elements within one).  A tensor that does not fit (its device, type, shape
or strides) raises ``KtError`` with ``KT_ERR_INVALID`` before anything is launched, as the
library's own refusals do.  Nothing is computed here, and outputs are the caller's tensors.
Work goes to torch's current stream of the tensors' device unless ``stream`` names another;
tensors that other streams still use are the caller's to order, as with any torch call.
"""
from __future__ import annotations

import ctypes

import torch

from . import kt_mlp
from .kt_mlp import KT_ACT_GEGLU, KT_ACT_NONE, KT_BF16, KT_ERR_INVALID, KT_F16, KtError, _check

_VP, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float

KT_LAYERNORM_MAX_D = 16384
KT_LINEAR_I8_DOT_ROWS = 16
KT_MOE_MAX_TOKENS, KT_MOE_MAX_EXPERTS, KT_MOE_MAX_TOP_K = 64, 256, 16


class kt_moe_options(ctypes.Structure):
    _fields_ = [(n, _I64) for n in ("max_tokens", "D", "F", "experts", "top_k")] + \
               [(n, ctypes.c_int32) for n in ("act", "dtype", "bias", "normalize")]


class kt_moe_tensors(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("X", _VP), ("ldx", _I64)] + \
               [(n, _VP) for n in ("W_router", "W_up", "W_down", "b_up", "b_down", "R", "Y", "ids", "weights")]


# every entry point declared in include/kt_ops.h, with its ctypes signature
SIGNATURES = {
    "kt_layernorm_forward": ([_I64, _I64, _I32, _VP, _I64, _VP, _VP, _F32, _VP, _I64, _VP, _VP, _VP], _I32),
    "kt_layernorm_backward": ([_I64, _I64, _I32, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _I64, _VP, _VP, _VP,
                               ctypes.c_size_t, _VP], _I32),
    "kt_layernorm_backward_workspace": ([_I64, _I64], ctypes.c_size_t),
    "kt_quantize_rows": ([_I64, _I64, _I32, _I32, _VP, _I64, _VP, _I64, _VP, _VP], _I32),
    "kt_linear_i8": ([_I64, _I64, _I64, _I32, _VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _I64, _VP], _I32),
    "kt_moe_plan": ([ctypes.POINTER(kt_moe_options), ctypes.POINTER(_VP)], _I32),
    "kt_moe_run": ([_VP, ctypes.POINTER(kt_moe_tensors), _VP], _I32),
    "kt_moe_status": ([_VP], _I32),
    "kt_moe_destroy": ([_VP], _I32),
}

_DTYPES = {torch.float16: KT_F16, torch.bfloat16: KT_BF16}
_F32_T, _I8_T, _I32_T = torch.float32, torch.int8, torch.int32
_lib = None
_fwd = _bwd = _quant = _lin = _moe = None  # the functions of the hot calls, once loaded


def load():
    """The shared library with this header's signatures set (``OSError`` if it has not been built)."""
    global _lib, _fwd, _bwd, _quant, _lin, _moe
    if _lib is None:
        lib = kt_mlp.load()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _fwd, _bwd, _quant = lib.kt_layernorm_forward, lib.kt_layernorm_backward, lib.kt_quantize_rows
        _lin, _moe = lib.kt_linear_i8, lib.kt_moe_run
        _lib = lib
    return _lib


def _bad(where: str, message: str):
    raise KtError(KT_ERR_INVALID, where, message)


def _size(where: str, name: str, t):
    """(rows, columns, device index) of a matrix."""
    shape = t.shape
    if len(shape) != 2:
        _bad(where, f"{name}: a matrix expected, got {list(shape)}")
    return shape[0], shape[1], t.get_device()


def _dtype(where: str, t) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        _bad(where, f"float16 or bfloat16 expected, got {t.dtype}")
    return code


def _rows(where: str, name: str, t, shape, dtype, index) -> int:
    """Checks a matrix with consecutive elements in a row; returns its row pitch."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        _bad(where, f"{name}: expected {dtype} {list(shape)} on device {index}, got {t.dtype} {list(t.shape)} on {t.device}")
    s0, s1 = t.stride()
    rows, cols = shape
    if s1 != 1 and cols > 1:
        _bad(where, f"{name}: elements of a row must be consecutive, strides are {t.stride()}")
    if s0 < cols:
        if rows > 1:
            _bad(where, f"{name}: rows overlap, strides are {t.stride()}")
        return cols  # the pitch of a single row is never used
    return s0


def _whole(where: str, name: str, t, shape, dtype, index) -> int:
    """Checks a contiguous tensor of the given shape; returns its address."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _bad(where, f"{name}: expected a contiguous {dtype} tensor {list(shape)} on device {index}, got {t.dtype} "
                    f"{list(t.shape)} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _on(where: str, index: int, stream) -> int:
    """The stream to launch on; the tensors' device must be the current one."""
    if index < 0:
        _bad(where, "CUDA tensors expected")
    if index != torch._C._cuda_getDevice():
        _bad(where, f"the tensors are on cuda:{index}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def kt_layernorm_forward(X, gamma, beta, eps, Y, mean=None, rstd=None, stream=None) -> None:
    """Y = layer norm of the rows of X; mean and rstd (fp32 [M]) receive the statistics if given."""
    w = "kt_layernorm_forward"
    M, D, dev = _size(w, "X", X)
    code, dt = _dtype(w, X), X.dtype
    s = _on(w, dev, stream)
    ldx, ldy = _rows(w, "X", X, (M, D), dt, dev), _rows(w, "Y", Y, (M, D), dt, dev)
    if _fwd is None:
        load()
    status = _fwd(M, D, code, X.data_ptr(), ldx, None if gamma is None else _whole(w, "gamma", gamma, (D,), dt, dev),
                  None if beta is None else _whole(w, "beta", beta, (D,), dt, dev), eps, Y.data_ptr(), ldy,
                  None if mean is None else _whole(w, "mean", mean, (M,), _F32_T, dev),
                  None if rstd is None else _whole(w, "rstd", rstd, (M,), _F32_T, dev), s)
    if status:
        _check(status, w)


def kt_layernorm_backward_workspace(M: int, D: int) -> int:
    """Bytes of workspace of kt_layernorm_backward (0 for sizes that it refuses)."""
    return load().kt_layernorm_backward_workspace(M, D)


def layernorm_backward_workspace(M: int, D: int, device="cuda"):
    """A workspace tensor for kt_layernorm_backward, to be kept from call to call on one stream."""
    return torch.empty(kt_layernorm_backward_workspace(M, D), dtype=torch.uint8, device=device)


def kt_layernorm_backward(dY, X, gamma, mean, rstd, dX, dgamma=None, dbeta=None, workspace=None, stream=None) -> None:
    """dX, and with dgamma and dbeta (fp32 [D]) their sums over the rows, which need ``workspace``
    (``layernorm_backward_workspace``)."""
    w = "kt_layernorm_backward"
    M, D, dev = _size(w, "X", X)
    code, dt, shape = _dtype(w, X), X.dtype, (M, D)
    s = _on(w, dev, stream)
    ldx, lddy, lddx = _rows(w, "X", X, shape, dt, dev), _rows(w, "dY", dY, shape, dt, dev), _rows(w, "dX", dX, shape, dt, dev)
    size = at = 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _bad(w, f"workspace: a contiguous tensor on device {dev} expected")
        size, at = workspace.nbytes, workspace.data_ptr()
    if _bwd is None:
        load()
    status = _bwd(M, D, code, dY.data_ptr(), lddy, X.data_ptr(), ldx,
                  None if gamma is None else _whole(w, "gamma", gamma, (D,), dt, dev),
                  _whole(w, "mean", mean, (M,), _F32_T, dev), _whole(w, "rstd", rstd, (M,), _F32_T, dev), dX.data_ptr(), lddx,
                  None if dgamma is None else _whole(w, "dgamma", dgamma, (D,), _F32_T, dev),
                  None if dbeta is None else _whole(w, "dbeta", dbeta, (D,), _F32_T, dev), at, size, s)
    if status:
        _check(status, w)


def kt_quantize_rows(X, Q, scale, act: int = KT_ACT_NONE, stream=None) -> None:
    """Q (int8 [M][K]) and scale (fp32 [M]) of act(X); X is [M][K], or [M][2K] for KT_ACT_GEGLU."""
    w = "kt_quantize_rows"
    M, K, dev = _size(w, "Q", Q)
    code = _dtype(w, X)
    s = _on(w, dev, stream)
    ldx = _rows(w, "X", X, (M, 2 * K if act == KT_ACT_GEGLU else K), X.dtype, dev)
    ldq = _rows(w, "Q", Q, (M, K), _I8_T, dev)
    if _quant is None:
        load()
    status = _quant(M, K, code, act, X.data_ptr(), ldx, Q.data_ptr(), ldq, _whole(w, "scale", scale, (M,), _F32_T, dev), s)
    if status:
        _check(status, w)


def kt_linear_i8(Q, scale_x, W, scale_w, bias, Y, stream=None) -> None:
    """Y[m][n] = scale_x[m] scale_w[n] sum_k Q[m][k] W[n][k] (+ bias[n])."""
    w = "kt_linear_i8"
    M, K, dev = _size(w, "Q", Q)
    N = _size(w, "W", W)[0]
    code, dt = _dtype(w, Y), Y.dtype
    s = _on(w, dev, stream)
    ldq, ldw, ldy = _rows(w, "Q", Q, (M, K), _I8_T, dev), _rows(w, "W", W, (N, K), _I8_T, dev), _rows(w, "Y", Y, (M, N), dt, dev)
    if M <= 1:
        ldq = (ldq + 15) // 16 * 16  # the pitch of a single row is never used
    if N <= 1:
        ldw = (ldw + 15) // 16 * 16
    if _lin is None:
        load()
    status = _lin(M, N, K, code, Q.data_ptr(), ldq, W.data_ptr(), ldw, _whole(w, "scale_x", scale_x, (M,), _F32_T, dev),
                  _whole(w, "scale_w", scale_w, (N,), _F32_T, dev),
                  None if bias is None else _whole(w, "bias", bias, (N,), dt, dev), Y.data_ptr(), ldy, s)
    if status:
        _check(status, w)


def kt_moe_plan(options: kt_moe_options) -> int:
    out = _VP()
    _check(load().kt_moe_plan(ctypes.byref(options), ctypes.byref(out)), "kt_moe_plan")
    return out.value


def kt_moe_run(plan: int, tensors: kt_moe_tensors, stream=None) -> None:
    if _moe is None:
        load()
    status = _moe(plan, ctypes.byref(tensors), kt_mlp._stream(stream))
    if status:
        _check(status, "kt_moe_run")


def kt_moe_status(plan: int) -> int:
    """Returns the status code (does not raise on KT_ERR_TIMEOUT)."""
    return load().kt_moe_status(plan)


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
        self.torch_dtype = torch.float16 if dtype == KT_F16 else torch.bfloat16

    def run(self, X, W_router, W_up, W_down, Y, b_up=None, b_down=None, R=None, ids=None, weights=None, stream=None):
        w, dt = "kt_moe_run", self.torch_dtype
        T, D, dev = _size(w, "X", X)
        E, shape, chosen = self.experts, (T, self.D), (T, self.top_k)
        s = _on(w, dev, stream)
        ldx = _rows(w, "X", X, shape, dt, dev)
        if T <= 1:
            ldx = (ldx + 7) // 8 * 8  # the pitch of a single row is never used
        kt_moe_run(self.handle, kt_moe_tensors(
            T, X.data_ptr(), ldx, _whole(w, "W_router", W_router, (E, D), dt, dev),
            _whole(w, "W_up", W_up, (E, self.rows, D), dt, dev), _whole(w, "W_down", W_down, (E, D, self.F), dt, dev),
            None if b_up is None else _whole(w, "b_up", b_up, (E, self.rows), dt, dev),
            None if b_down is None else _whole(w, "b_down", b_down, (E, D), dt, dev),
            None if R is None else _whole(w, "R", R, shape, dt, dev), _whole(w, "Y", Y, shape, dt, dev),
            None if ids is None else _whole(w, "ids", ids, chosen, _I32_T, dev),
            None if weights is None else _whole(w, "weights", weights, chosen, _F32_T, dev)), s)

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
