"""The operators of a training step and of serving in 8-bit floating point, on the CPU: their refusals (every check
precedes the device query, so none needs a GPU), and the formulas of the gradients against differences."""
import ctypes

import pytest
import torch

from transformer_mlp_gemms_gb300 import build as kbuild
from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops

import train_reference as ref

INVALID, UNSUPPORTED = kt_mlp.KT_ERR_INVALID, kt_mlp.KT_ERR_UNSUPPORTED
P = 1 << 20  # an address that is aligned to anything; no refused call reads it


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kt_ops.load()


SIZES = [(dict(M=-1), INVALID), (dict(D=0), INVALID), (dict(F=0), INVALID), (dict(dtype=2), INVALID), (dict(act=6), INVALID),
         (dict(act=2), INVALID), (dict(ldx=32), INVALID), (dict(X=P + 8), INVALID), (dict(X=None), INVALID), (dict(W=None), INVALID),
         (dict(W=P + 2), INVALID), (dict(ldx=68), UNSUPPORTED), (dict(D=60, ldx=64), UNSUPPORTED), (dict(F=36), UNSUPPORTED),
         (dict(M=1 << 31), UNSUPPORTED), (dict(ldp=72), INVALID), (dict(ldp=84), UNSUPPORTED), (dict(P=P + 4), INVALID)]
FWD = dict(M=4, D=64, F=40, dtype=0, act=5, X=P, ldx=64, W=P, b=P, H=P, ldh=40, P=P, ldp=80)


@pytest.mark.parametrize("kw,status", SIZES + [(dict(H=None), INVALID), (dict(ldh=32), INVALID), (dict(ldh=44), UNSUPPORTED), (dict(b=P + 8), INVALID)])
def test_glu_forward_refusals(lib, kw, status):
    a = {**FWD, **kw}
    got = lib.kt_glu_forward(a["M"], a["D"], a["F"], a["dtype"], a["act"], a["X"], a["ldx"], a["W"], a["b"], a["H"], a["ldh"], a["P"],
                             a["ldp"], None)
    assert got == status and kt_mlp.kt_last_error()


BWD = dict(M=4, D=64, F=40, dtype=0, act=5, dH=P, lddh=40, P=P, ldp=80, X=P, ldx=64, W=P, dX=P, lddx=64, dW=P, db=P, ws=P, size=1 << 20)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(dH=None), INVALID), (dict(P=None), INVALID), (dict(lddh=32), INVALID), (dict(lddx=32), INVALID), (dict(lddx=68), UNSUPPORTED),
    (dict(dX=P + 2), INVALID), (dict(dW=P + 8), INVALID), (dict(db=P + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=P + 8), INVALID),
    (dict(size=64), INVALID)])
def test_glu_backward_refusals(lib, kw, status):
    a = {**BWD, **kw}
    got = lib.kt_glu_backward(a["M"], a["D"], a["F"], a["dtype"], a["act"], a["dH"], a["lddh"], a["P"], a["ldp"], a["X"], a["ldx"], a["W"],
                              a["dX"], a["lddx"], a["dW"], a["db"], a["ws"], a["size"], None)
    assert got == status and kt_mlp.kt_last_error()


LIN = dict(M=4, N=40, K=64, dtype=1, X=P, ldx=64, W=P, b=None, Y=P, ldy=40, dX=P, lddx=64, dW=P, db=P, ws=P, size=1 << 20)
LINEAR = [(dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(dtype=-1), INVALID), (dict(X=None), INVALID),
          (dict(W=None), INVALID), (dict(Y=None), INVALID), (dict(ldx=56), INVALID), (dict(ldy=32), INVALID), (dict(X=P + 8), INVALID),
          (dict(Y=P + 8), INVALID), (dict(N=44, ldy=48), UNSUPPORTED), (dict(K=62), UNSUPPORTED), (dict(ldx=70), UNSUPPORTED),
          (dict(ldy=42), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", LINEAR + [(dict(b=P + 2), INVALID)])
def test_linear_forward_refusals(lib, kw, status):
    a = {**LIN, **kw}
    got = lib.kt_linear_forward(a["M"], a["N"], a["K"], a["dtype"], a["X"], a["ldx"], a["W"], a["b"], a["Y"], a["ldy"], None)
    assert got == status and kt_mlp.kt_last_error()


@pytest.mark.parametrize("kw,status", LINEAR + [(dict(lddx=56), INVALID), (dict(dX=P + 8), INVALID), (dict(dW=P + 8), INVALID),
                                                (dict(db=P + 1), INVALID), (dict(ws=None), INVALID), (dict(size=4), INVALID)])
def test_linear_backward_refusals(lib, kw, status):
    a = {**LIN, **kw}
    got = lib.kt_linear_backward(a["M"], a["N"], a["K"], a["dtype"], a["Y"], a["ldy"], a["X"], a["ldx"], a["W"], a["dX"], a["lddx"], a["dW"],
                                 a["db"], a["ws"], a["size"], None)
    assert got == status and kt_mlp.kt_last_error()


def test_workspace_sizes(lib):
    glu, linear = lib.kt_glu_backward_workspace, lib.kt_linear_backward_workspace
    assert glu(-1, 64, 64) == glu(4, 0, 64) == glu(4, 64, 60) == glu(1 << 31, 64, 64) == 0
    assert linear(-1, 64, 64) == linear(4, 4, 64) == linear(4, 64, 0) == 0
    assert glu(0, 64, 64) >= 2 * 64 * 4 and linear(0, 64, 64) >= 64 * 4
    assert glu(1000, 64, 64) >= 1000 * 2 * 64 * 2 + 2 * 64 * 4
    assert linear(1 << 20, 64, 64) <= 128 * 64 * 4 + (42 << 20)  # partial sums of at most 80 pairs of CTAs, two tiles each


def adamw(lib, tensor, options, count=1):
    t = kt_ops.kt_adamw_tensor(**{**dict(param=P, grad=P, m=P + 4096, v=P + 8192, m_scale=None, v_scale=None, copy=None, n=100, weight_decay=0.0), **tensor})
    o = kt_ops.kt_adamw_options(**{**dict(param_dtype=2, grad_dtype=1, copy_dtype=1, state_bits=32, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8,
                                          step=1, step_device=None, grad_scale=None), **options})
    return lib.kt_adamw(count, ctypes.byref(t), ctypes.byref(o), None)


@pytest.mark.parametrize("tensor,options", [
    (dict(param=None), {}), (dict(grad=None), {}), (dict(m=None), {}), (dict(v=None), {}), (dict(n=-1), {}), (dict(param=P + 2), {}),
    (dict(grad=P + 1), {}), (dict(m=P + 2), {}), (dict(copy=P + 1), {}), (dict(weight_decay=float("inf")), {}),
    (dict(weight_decay=float("nan")), {}), (dict(copy=P), dict(param_dtype=1)), (dict(copy=P), dict(copy_dtype=2)), ({}, dict(param_dtype=3)),
    ({}, dict(grad_dtype=-1)), ({}, dict(state_bits=16)), ({}, dict(state_bits=8)), ({}, dict(lr=-1.0)), ({}, dict(lr=float("nan"))),
    ({}, dict(eps=float("inf"))), ({}, dict(beta1=1.0)), ({}, dict(beta2=-0.1)), ({}, dict(beta2=float("nan"))), ({}, dict(step=0)),
    ({}, dict(step_device=P + 4)), ({}, dict(grad_scale=P + 2)), (dict(m=P), {}), (dict(v=P + 4096), {}),
])
def test_adamw_refusals(lib, tensor, options):
    assert adamw(lib, tensor, options) == INVALID and kt_mlp.kt_last_error()


@pytest.mark.parametrize("count", [2, 64, 65, 400])
def test_adamw_refuses_tied_parameters(lib, count):
    o = kt_ops.kt_adamw_options(param_dtype=2, grad_dtype=2, state_bits=32, lr=1e-3, beta1=0.9, beta2=0.99, eps=0.0, step=1)
    tensors = (kt_ops.kt_adamw_tensor * count)()
    for i, t in enumerate(tensors):
        t.n = 4
        t.param, t.grad, t.m, t.v = (P + 1024 * (4 * i + j) for j in range(4))
    tensors[count - 1].param = tensors[0].param
    assert lib.kt_adamw(count, tensors, ctypes.byref(o), None) == INVALID and "twice" in kt_mlp.kt_last_error()
    tensors[0].n = 0  # an empty tensor is not updated
    assert lib.kt_adamw(count, tensors, ctypes.byref(o), None) != INVALID


def test_adamw_without_tensors(lib):
    o = kt_ops.kt_adamw_options(param_dtype=2, grad_dtype=2, state_bits=32, lr=1e-3, beta1=0.9, beta2=0.99, eps=0.0, step=1)
    assert lib.kt_adamw(0, None, ctypes.byref(o), None) == kt_mlp.KT_OK
    assert adamw(lib, dict(n=0, param=None, grad=None, m=None, v=None), {}) == kt_mlp.KT_OK
    assert lib.kt_adamw(1, None, ctypes.byref(o), None) == INVALID
    assert lib.kt_adamw(-1, None, ctypes.byref(o), None) == INVALID
    assert lib.kt_adamw(0, None, None, None) == INVALID


Q = dict(M=4, K=64, dtype=0, act=3, X=P, ldx=64, Q=P, ldq=64, scale=P)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(dtype=2), INVALID), (dict(act=6), INVALID), (dict(ldx=32), INVALID),
    (dict(act=2), INVALID), (dict(ldq=32), INVALID), (dict(X=None), INVALID), (dict(Q=None), INVALID), (dict(scale=None), INVALID),
    (dict(scale=P + 2), INVALID), (dict(X=P + 1), INVALID), (dict(M=1 << 31), UNSUPPORTED),
])
def test_quantize_fp8_refusals(lib, kw, status):
    a = {**Q, **kw}
    got = lib.kt_quantize_fp8(a["M"], a["K"], a["dtype"], a["act"], a["X"], a["ldx"], a["Q"], a["ldq"], a["scale"], None)
    assert got == status and kt_mlp.kt_last_error()


F8 = dict(M=4, N=8, K=64, dtype=0, Q=P, ldq=64, W=P, ldw=64, sx=P, sw=P, bias=None, Y=P, ldy=8)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(dtype=2), INVALID), (dict(ldq=32), INVALID),
    (dict(ldw=32), INVALID), (dict(ldy=4), INVALID), (dict(Q=None), INVALID), (dict(W=None), INVALID), (dict(sx=None), INVALID),
    (dict(sw=None), INVALID), (dict(Y=None), INVALID), (dict(Q=P + 8), INVALID), (dict(W=P + 4), INVALID), (dict(Y=P + 2), INVALID),
    (dict(bias=P + 2), INVALID), (dict(sx=P + 2), INVALID), (dict(K=40), UNSUPPORTED), (dict(ldq=72), UNSUPPORTED),
    (dict(ldw=68), UNSUPPORTED), (dict(N=12, ldy=16), UNSUPPORTED), (dict(ldy=12), UNSUPPORTED),
])
def test_linear_fp8_refusals(lib, kw, status):
    a = {**F8, **kw}
    got = lib.kt_linear_fp8(a["M"], a["N"], a["K"], a["dtype"], a["Q"], a["ldq"], a["W"], a["ldw"], a["sx"], a["sw"], a["bias"], a["Y"],
                            a["ldy"], None)
    assert got == status and kt_mlp.kt_last_error()


@pytest.mark.parametrize("limit_us", [0, -1, 10_000_001])
def test_debug_stall_refuses_a_limit(lib, limit_us):
    assert lib.kt_matmul_debug_stall(1, limit_us) == INVALID
    assert lib.kt_matmul_debug_stall(0, limit_us) == kt_mlp.KT_OK


def test_without_a_gpu_nothing_is_computed(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    refused = (kt_mlp.KT_ERR_CUDA, UNSUPPORTED)
    assert lib.kt_linear_forward(4, 8, 64, 0, P, 64, P, None, P, 8, None) in refused
    assert adamw(lib, {}, {}) in refused
    assert lib.kt_matmul_status(None) in refused


def test_tensors_that_do_not_fit_are_refused_by_the_binding():
    h = torch.float16
    x, w = torch.zeros(4, 64, dtype=h), torch.zeros(80, 64, dtype=h)
    H, P_, f = torch.zeros(4, 40, dtype=h), torch.zeros(4, 80, dtype=h), torch.zeros(100)
    e4 = lambda *s: torch.zeros(*s, dtype=torch.float8_e4m3fn)  # noqa: E731
    glu = lambda **k: kt_ops.kt_glu_forward(**{**dict(X=x, W=w, bias=None, H=H, P=P_, act=5), **k})  # noqa: E731
    adam = lambda **k: kt_ops.kt_adamw(**{**dict(params=[f], grads=[f], m=[f], v=[f], step=1, lr=1e-3), **k})  # noqa: E731
    cases = [
        lambda: glu(),                                                # not on a GPU
        lambda: glu(W=None), lambda: glu(W=w[:40]), lambda: glu(W=w.t()), lambda: glu(W=w.float()), lambda: glu(bias=w[0]),
        lambda: glu(H=H[:3]), lambda: glu(P=H), lambda: glu(X=x.float()), lambda: glu(H=H.bfloat16()), lambda: glu(act="silu"),
        lambda: kt_ops.kt_glu_backward(H, P_, x, w, x, w[:8], None, 5, torch.zeros(8)),
        lambda: kt_ops.kt_glu_backward(H, P_, x, w, x, w, torch.zeros(80, dtype=h), 5, torch.zeros(8)),
        lambda: kt_ops.kt_linear_forward(x, w, None, H),
        lambda: kt_ops.kt_linear_backward(P_, x, w, x, w, torch.zeros(80), None),
        lambda: adam(grads=[]), lambda: adam(m=[f[:9]]), lambda: adam(params=[f.half()], copies=[f.half()]), lambda: adam(m=[f.half()]),
        lambda: adam(m=[e4(100)], v=[e4(100)]), lambda: adam(m_scales=[f[:1]], v_scales=[f[:1]]), lambda: adam(params=f),
        lambda: adam(weight_decay="0"), lambda: adam(weight_decay=[0.1, 0.1]), lambda: adam(params=[torch.zeros(200)[::2]]),
        lambda: adam(step=torch.zeros(1)), lambda: adam(grads=[None]),
        lambda: kt_ops.kt_quantize_fp8(x, x, f[:4].view(4, 1)),
        lambda: kt_ops.kt_quantize_fp8(x, e4(4, 64), f[:8].view(4, 2)),
        lambda: kt_ops.kt_linear_fp8(e4(4, 64), f[:4].view(4, 1), e4(8, 32), f[:1].view(1, 1), None, torch.zeros(4, 8, dtype=h)),
    ]
    for i, call in enumerate(cases):
        with pytest.raises(kt_mlp.KtError) as e:
            call()
        assert e.value.status == INVALID, i


def differences(loss, tensors, grads, h=1e-5):
    """Central differences, off by h^2 f''' / 6 plus 2^-52 |f| / h: below 1e-8 for values around 1 and sums around 100."""
    for t, grad in zip(tensors, grads):
        flat = t.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            down = loss()
            flat[i] = keep
            assert abs((up - down) / (2 * h) - grad.reshape(-1)[i]) < 1e-7


@pytest.mark.parametrize("name", ["gelu_erf", "gelu_tanh", "gelu_sigmoid", "silu", "none"])
def test_gated_gradients_agree_with_differences(name):
    torch.manual_seed(1)
    M, D, F, d = 3, 4, 5, torch.float64
    x, w, b, dh = torch.randn(M, D, dtype=d), torch.randn(2 * F, D, dtype=d), torch.randn(2 * F, dtype=d), torch.randn(M, F, dtype=d)
    p = x @ w.t() + b
    dx, _, dw, _, db, _ = ref.glu_backward(dh, p, x, w, name, torch.float16)
    differences(lambda: (ref.glu(x, w, b, name, torch.float16)[0] * dh).sum(), (x, w, b), (dx, dw, db))


def test_linear_gradients_agree_with_differences():
    torch.manual_seed(2)
    M, N, K, d = 3, 4, 5, torch.float64
    x, w, b, dy = torch.randn(M, K, dtype=d), torch.randn(N, K, dtype=d), torch.randn(N, dtype=d), torch.randn(M, N, dtype=d)
    dx, _, dw, _, db, _ = ref.linear_backward(dy, x, w, torch.float16)
    differences(lambda: (ref.product(x, w, b)[0] * dy).sum(), (x, w, b), (dx, dw, db))
