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
from .kt_mlp import KT_ACT_GEGLU, KT_ACT_NONE, KT_BF16, KT_ERR_INVALID, KT_F16, KtError, _check, _ptr

_VP, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float

KT_LAYERNORM_MAX_D = 16384
KT_LINEAR_I8_DOT_ROWS = 8
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
_lib = None


def load():
    """The shared library with this header's signatures set (``OSError`` if it has not been built)."""
    global _lib
    if _lib is None:
        lib = kt_mlp.load()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _bad(where: str, message: str):
    raise KtError(KT_ERR_INVALID, where, message)


def _dtype(where: str, t) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        _bad(where, f"float16 or bfloat16 expected, got {t.dtype}")
    return code


def _matrix(where: str, name: str, t, rows, cols, dtype, device) -> int:
    """Checks a [rows][cols] tensor with consecutive elements in a row; returns its row pitch."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        _bad(where, f"{name}: expected [{rows}][{cols}], got {list(t.shape)}")
    if t.dtype != dtype or t.device != device:
        _bad(where, f"{name}: expected {dtype} on {device}, got {t.dtype} on {t.device}")
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        _bad(where, f"{name}: elements of a row must be consecutive, strides are {t.stride()}")
    if rows <= 1:
        return max(s0, cols)
    if s0 < cols:
        _bad(where, f"{name}: rows overlap, strides are {t.stride()}")
    return s0


def _whole(where: str, name: str, t, shape, dtype, device):
    """Checks a contiguous tensor of the given shape."""
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        _bad(where, f"{name}: expected a contiguous {dtype} tensor {list(shape)} on {device}, got {t.dtype} "
                    f"{list(t.shape)} on {t.device}, strides {t.stride()}")


def _on(where: str, device, stream):
    """The stream to launch on; the tensors' device must be the current one."""
    if device.type != "cuda":
        _bad(where, f"CUDA tensors expected, got {device}")
    if device.index != torch.cuda.current_device():
        _bad(where, f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def kt_layernorm_forward(X, gamma, beta, eps, Y, mean=None, rstd=None, stream=None) -> None:
    """Y = layer norm of the rows of X; mean and rstd (fp32 [M]) receive the statistics if given."""
    w = "kt_layernorm_forward"
    if X.dim() != 2:
        _bad(w, f"X: a matrix expected, got {list(X.shape)}")
    (M, D), dev, dt = X.shape, X.device, X.dtype
    code = _dtype(w, X)
    ldx, ldy = _matrix(w, "X", X, M, D, dt, dev), _matrix(w, "Y", Y, M, D, dt, dev)
    for name, t in (("gamma", gamma), ("beta", beta)):
        if t is not None:
            _whole(w, name, t, (D,), dt, dev)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _whole(w, name, t, (M,), torch.float32, dev)
    s = _on(w, dev, stream)
    _check(load().kt_layernorm_forward(M, D, code, X.data_ptr(), ldx, _ptr(gamma), _ptr(beta), eps, Y.data_ptr(), ldy,
                                       _ptr(mean), _ptr(rstd), s), w)


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
    if X.dim() != 2:
        _bad(w, f"X: a matrix expected, got {list(X.shape)}")
    (M, D), dev, dt = X.shape, X.device, X.dtype
    code = _dtype(w, X)
    ldx, lddy, lddx = (_matrix(w, n, t, M, D, dt, dev) for n, t in (("X", X), ("dY", dY), ("dX", dX)))
    if gamma is not None:
        _whole(w, "gamma", gamma, (D,), dt, dev)
    _whole(w, "mean", mean, (M,), torch.float32, dev)
    _whole(w, "rstd", rstd, (M,), torch.float32, dev)
    for name, t in (("dgamma", dgamma), ("dbeta", dbeta)):
        if t is not None:
            _whole(w, name, t, (D,), torch.float32, dev)
    size = 0
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            _bad(w, f"workspace: a contiguous tensor on {dev} expected")
        size = workspace.numel() * workspace.element_size()
    s = _on(w, dev, stream)
    _check(load().kt_layernorm_backward(M, D, code, dY.data_ptr(), lddy, X.data_ptr(), ldx, _ptr(gamma), mean.data_ptr(),
                                        rstd.data_ptr(), dX.data_ptr(), lddx, _ptr(dgamma), _ptr(dbeta), _ptr(workspace),
                                        size, s), w)


def kt_quantize_rows(X, Q, scale, act: int = KT_ACT_NONE, stream=None) -> None:
    """Q (int8 [M][K]) and scale (fp32 [M]) of act(X); X is [M][K], or [M][2K] for KT_ACT_GEGLU."""
    w = "kt_quantize_rows"
    if X.dim() != 2 or Q.dim() != 2:
        _bad(w, f"X and Q: matrices expected, got {list(X.shape)} and {list(Q.shape)}")
    M, K, dev = X.shape[0], Q.shape[1], X.device
    code = _dtype(w, X)
    ldx = _matrix(w, "X", X, M, 2 * K if act == KT_ACT_GEGLU else K, X.dtype, dev)
    ldq = _matrix(w, "Q", Q, M, K, torch.int8, dev)
    _whole(w, "scale", scale, (M,), torch.float32, dev)
    s = _on(w, dev, stream)
    _check(load().kt_quantize_rows(M, K, code, act, X.data_ptr(), ldx, Q.data_ptr(), ldq, scale.data_ptr(), s), w)


def kt_linear_i8(Q, scale_x, W, scale_w, bias, Y, stream=None) -> None:
    """Y[m][n] = scale_x[m] scale_w[n] sum_k Q[m][k] W[n][k] (+ bias[n])."""
    w = "kt_linear_i8"
    if Q.dim() != 2 or W.dim() != 2:
        _bad(w, f"Q and W: matrices expected, got {list(Q.shape)} and {list(W.shape)}")
    (M, K), N, dev = Q.shape, W.shape[0], Q.device
    code = _dtype(w, Y)
    ldq, ldw = _matrix(w, "Q", Q, M, K, torch.int8, dev), _matrix(w, "W", W, N, K, torch.int8, dev)
    ldy = _matrix(w, "Y", Y, M, N, Y.dtype, dev)
    _whole(w, "scale_x", scale_x, (M,), torch.float32, dev)
    _whole(w, "scale_w", scale_w, (N,), torch.float32, dev)
    if bias is not None:
        _whole(w, "bias", bias, (N,), Y.dtype, dev)
    if M <= 1:
        ldq = (ldq + 15) // 16 * 16  # the pitch of a single row is never used
    if N <= 1:
        ldw = (ldw + 15) // 16 * 16
    s = _on(w, dev, stream)
    _check(load().kt_linear_i8(M, N, K, code, Q.data_ptr(), ldq, W.data_ptr(), ldw, scale_x.data_ptr(),
                               scale_w.data_ptr(), _ptr(bias), Y.data_ptr(), ldy, s), w)


def kt_moe_plan(options: kt_moe_options) -> int:
    out = _VP()
    _check(load().kt_moe_plan(ctypes.byref(options), ctypes.byref(out)), "kt_moe_plan")
    return out.value


def kt_moe_run(plan: int, tensors: kt_moe_tensors, stream=None) -> None:
    _check(load().kt_moe_run(plan, ctypes.byref(tensors), kt_mlp._stream(stream)), "kt_moe_run")


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
        w, dt, dev = "kt_moe_run", self.torch_dtype, X.device
        if X.dim() != 2:
            _bad(w, f"X: a matrix expected, got {list(X.shape)}")
        T, D, E = X.shape[0], self.D, self.experts
        ldx = _matrix(w, "X", X, T, D, dt, dev)
        if T <= 1:
            ldx = (ldx + 7) // 8 * 8  # the pitch of a single row is never used
        _whole(w, "W_router", W_router, (E, D), dt, dev)
        _whole(w, "W_up", W_up, (E, self.rows, D), dt, dev)
        _whole(w, "W_down", W_down, (E, D, self.F), dt, dev)
        _whole(w, "Y", Y, (T, D), dt, dev)
        if b_up is not None:
            _whole(w, "b_up", b_up, (E, self.rows), dt, dev)
        if b_down is not None:
            _whole(w, "b_down", b_down, (E, D), dt, dev)
        if R is not None:
            _whole(w, "R", R, (T, D), dt, dev)
        if ids is not None:
            _whole(w, "ids", ids, (T, self.top_k), torch.int32, dev)
        if weights is not None:
            _whole(w, "weights", weights, (T, self.top_k), torch.float32, dev)
        s = _on(w, dev, stream)
        kt_moe_run(self.handle, kt_moe_tensors(T, X.data_ptr(), ldx, W_router.data_ptr(), W_up.data_ptr(),
                                               W_down.data_ptr(), _ptr(b_up), _ptr(b_down), _ptr(R), Y.data_ptr(),
                                               _ptr(ids), _ptr(weights)), s)

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
