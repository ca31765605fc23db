"""The operators around the MLP on the CPU: the boundary that include/kt_ops.h declares, its
refusals (every check precedes the device query, so none needs a GPU), and the formulas of the
gradients against differences."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

from transformer_mlp_gemms_gb300 import build as kbuild
from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops

import ops_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = kt_mlp.KT_ERR_INVALID, kt_mlp.KT_ERR_UNSUPPORTED
P = 1 << 20  # an address that is aligned to anything; no refused call reads it


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kt_ops.load()


def test_the_binding_wraps_what_the_header_declares(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kt_ops.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(kt_\w+)\s*\(", text))
    assert names == set(kt_ops.SIGNATURES)
    assert all(hasattr(lib, n) and hasattr(kt_ops, n) for n in names)


def test_limits_agree_with_the_header():
    text = open(os.path.join(ROOT, "include", "kt_ops.h")).read()
    for name, value in re.findall(r"#define (KT_\w+) (\d+)", text):
        assert getattr(kt_ops, name) == int(value), name


LN = dict(M=4, D=64, dtype=0, X=P, ldx=64, gamma=P, beta=P, eps=1e-5, Y=P * 2, ldy=64, mean=P, rstd=P)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(D=0), INVALID), (dict(dtype=2), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(gamma=None), INVALID), (dict(beta=None), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(X=P + 1), INVALID), (dict(mean=P + 2), INVALID), (dict(X=P * 2, ldx=72), INVALID),
    (dict(D=16385, ldx=16385, ldy=16385), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
])
def test_layernorm_forward_refusals(lib, kw, status):
    a = {**LN, **kw}
    got = lib.kt_layernorm_forward(a["M"], a["D"], a["dtype"], a["X"], a["ldx"], a["gamma"], a["beta"], a["eps"], a["Y"],
                                   a["ldy"], a["mean"], a["rstd"], None)
    assert got == status and kt_mlp.kt_last_error()


BWD = dict(M=4, D=64, dtype=1, dY=P, lddy=64, X=P * 2, ldx=64, gamma=P, mean=P, rstd=P, dX=P * 3, lddx=64, dgamma=P,
           dbeta=P, ws=P, size=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(D=0), INVALID), (dict(dtype=-1), INVALID), (dict(lddy=8), INVALID), (dict(lddx=8), INVALID),
    (dict(dY=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(dX=None), INVALID),
    (dict(dgamma=None), INVALID), (dict(dbeta=None), INVALID), (dict(ws=None), INVALID), (dict(size=8), INVALID),
    (dict(ws=P + 8), INVALID), (dict(dX=P, lddx=72), INVALID), (dict(D=20000, lddy=20000, ldx=20000, lddx=20000), UNSUPPORTED),
])
def test_layernorm_backward_refusals(lib, kw, status):
    a = {**BWD, **kw}
    got = lib.kt_layernorm_backward(a["M"], a["D"], a["dtype"], a["dY"], a["lddy"], a["X"], a["ldx"], a["gamma"], a["mean"],
                                    a["rstd"], a["dX"], a["lddx"], a["dgamma"], a["dbeta"], a["ws"], a["size"], None)
    assert got == status and kt_mlp.kt_last_error()


def test_backward_workspace_sizes(lib):
    ws = lib.kt_layernorm_backward_workspace
    assert ws(-1, 8) == ws(4, 0) == ws(4, 16385) == ws(1 << 31, 8) == 0
    assert ws(0, 8) >= 2 * 8 * 4 and ws(1, 8) >= 2 * 8 * 4
    assert ws(100000, 1280) <= 160 * 2 * 1280 * 4


Q = dict(M=4, K=64, dtype=0, act=3, X=P, ldx=64, Q=P, ldq=64, scale=P)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(dtype=2), INVALID), (dict(act=6), INVALID), (dict(ldx=32), INVALID),
    (dict(act=2), INVALID), (dict(ldq=32), INVALID), (dict(X=None), INVALID), (dict(Q=None), INVALID), (dict(scale=None), INVALID),
    (dict(scale=P + 2), INVALID), (dict(K=20000, ldx=20000, ldq=20000), UNSUPPORTED),
])
def test_quantize_refusals(lib, kw, status):
    a = {**Q, **kw}
    got = lib.kt_quantize_rows(a["M"], a["K"], a["dtype"], a["act"], a["X"], a["ldx"], a["Q"], a["ldq"], a["scale"], None)
    assert got == status and kt_mlp.kt_last_error()


LIN = dict(M=4, N=8, K=64, dtype=0, Q=P, ldq=64, W=P, ldw=64, sx=P, sw=P, bias=None, Y=P, ldy=8)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(dtype=2), INVALID), (dict(ldq=32), INVALID),
    (dict(ldw=32), INVALID), (dict(ldy=4), INVALID), (dict(Q=None), INVALID), (dict(W=None), INVALID), (dict(sx=None), INVALID),
    (dict(Q=P + 8), INVALID), (dict(W=P + 4), INVALID), (dict(Y=P + 1), INVALID), (dict(bias=P + 1), INVALID),
    (dict(K=40), UNSUPPORTED), (dict(ldq=72), UNSUPPORTED), (dict(ldw=68), UNSUPPORTED),
    (dict(K=1 << 17, ldq=1 << 17, ldw=1 << 17), UNSUPPORTED),
])
def test_linear_i8_refusals(lib, kw, status):
    a = {**LIN, **kw}
    got = lib.kt_linear_i8(a["M"], a["N"], a["K"], a["dtype"], a["Q"], a["ldq"], a["W"], a["ldw"], a["sx"], a["sw"], a["bias"],
                           a["Y"], a["ldy"], None)
    assert got == status and kt_mlp.kt_last_error()


MOE = dict(max_tokens=4, D=64, F=64, experts=8, top_k=2, act=0, dtype=0, bias=0, normalize=1)


@pytest.mark.parametrize("kw,status", [
    (dict(max_tokens=0), INVALID), (dict(D=0), INVALID), (dict(F=-8), INVALID), (dict(experts=0), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=9), INVALID), (dict(act=6), INVALID), (dict(dtype=2), INVALID), (dict(bias=2), INVALID), (dict(normalize=-1), INVALID),
    (dict(max_tokens=65), UNSUPPORTED), (dict(experts=257), UNSUPPORTED), (dict(experts=32, top_k=17), UNSUPPORTED),
    (dict(D=60), UNSUPPORTED), (dict(F=12), UNSUPPORTED), (dict(D=65544), UNSUPPORTED),
])
def test_moe_plan_refusals(lib, kw, status):
    with pytest.raises(kt_mlp.KtError) as e:
        kt_ops.kt_moe_plan(kt_ops.kt_moe_options(**{**MOE, **kw}))
    assert e.value.status == status


def test_moe_null_handles(lib):
    out = ctypes.c_void_p()
    assert lib.kt_moe_plan(None, ctypes.byref(out)) == INVALID
    assert lib.kt_moe_plan(ctypes.byref(kt_ops.kt_moe_options(**MOE)), None) == INVALID
    assert lib.kt_moe_run(None, None, None) == INVALID
    assert lib.kt_moe_status(None) == INVALID
    assert lib.kt_moe_destroy(None) == INVALID


def test_without_a_gpu_nothing_is_computed(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    got = lib.kt_layernorm_forward(4, 64, 0, P, 64, P, P, 1e-5, 2 * P, 64, P, P, None)
    assert got in (kt_mlp.KT_ERR_CUDA, UNSUPPORTED)
    with pytest.raises(kt_mlp.KtError):
        kt_ops.MoePlan(4, 64, 64, 8, 2, 0, 0)


def test_tensors_that_do_not_fit_are_refused_by_the_binding():
    x = torch.zeros(4, 64, dtype=torch.float16)
    f = torch.zeros(4)
    cases = [
        lambda: kt_ops.kt_layernorm_forward(x, None, None, 1e-5, x),                          # not on a GPU
        lambda: kt_ops.kt_layernorm_forward(x.float(), None, None, 1e-5, x.float()),          # dtype
        lambda: kt_ops.kt_layernorm_forward(x, None, None, 1e-5, torch.zeros_like(x).t()),    # shape
        lambda: kt_ops.kt_layernorm_forward(x.t(), None, None, 1e-5, x.t()),                  # strides
        lambda: kt_ops.kt_layernorm_forward(x[:1].expand(4, 64), None, None, 1e-5, x),        # overlapping rows
        lambda: kt_ops.kt_layernorm_forward(x, x[0].float(), x[0], 1e-5, x),                  # gamma's dtype
        lambda: kt_ops.kt_layernorm_forward(x, None, None, 1e-5, x, mean=f.double()),         # statistics' dtype
        lambda: kt_ops.kt_layernorm_backward(x, x, None, f[:3], f, x),                        # statistics' length
        lambda: kt_ops.kt_quantize_rows(x, torch.zeros(4, 32, dtype=torch.int8), f),          # widths
        lambda: kt_ops.kt_linear_i8(torch.zeros(4, 64, dtype=torch.int8), f, torch.zeros(8, 32, dtype=torch.int8),
                                    torch.zeros(8), None, torch.zeros(4, 8, dtype=torch.float16)),
    ]
    for call in cases:
        with pytest.raises(kt_mlp.KtError) as e:
            call()
        assert e.value.status == INVALID


@pytest.mark.parametrize("affine", [True, False])
def test_gradient_formulas_agree_with_differences(affine):
    """The 64-bit formulas that the GPU tests compare with, against central differences of the
    forward formula.  For a smooth function the difference quotient is off by h^2 f'''/6 plus
    about 2^-52 |f| / h: with h = 1e-4 and |f| below 100, some 1e-8 to 1e-7 here."""
    torch.manual_seed(0)
    M, D, h = 3, 7, 1e-4
    x, dy = torch.randn(M, D, dtype=torch.float64), torch.randn(M, D, dtype=torch.float64)
    gamma, beta = torch.randn(D, dtype=torch.float64), torch.randn(D, dtype=torch.float64)
    if not affine:
        gamma, beta = torch.ones_like(gamma), torch.zeros_like(beta)

    def loss(x, gamma, beta):
        return (ref.layernorm(x, gamma, beta, 1e-5)[0] * dy).sum()

    _, mean, rstd = ref.layernorm(x, gamma, beta, 1e-5)
    dx, dgamma, dbeta = ref.layernorm_backward(dy, x, gamma, mean, rstd)
    for t, grad in ((x, dx), (gamma, dgamma), (beta, dbeta)):
        flat = t.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(x, gamma, beta)
            flat[i] = keep - h
            down = loss(x, gamma, beta)
            flat[i] = keep
            assert abs((up - down) / (2 * h) - grad.reshape(-1)[i]) < 1e-6


@pytest.mark.parametrize("limit_us", [0, -1, 10_000_001])
def test_linear_i8_debug_stall_refuses_a_limit(lib, limit_us):
    assert lib.kt_linear_i8_debug_stall(1, limit_us) == INVALID
    assert lib.kt_linear_i8_debug_stall(0, limit_us) == kt_mlp.KT_OK


def test_linear_i8_status_without_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lib.kt_linear_i8_status(None) in (kt_mlp.KT_ERR_CUDA, UNSUPPORTED)


def test_moe_debug_stall_refuses_a_null_plan(lib):
    assert lib.kt_moe_debug_stall(None, 1, 1000) == INVALID


def test_the_library_builds_without_torch(lib, tmp_path):
    """A C user of the headers needs nvcc alone: no torch, and so no module."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from transformer_mlp_gemms_gb300 import build as b\n"
            f"b.MODULE = {str(tmp_path / '_kt_ops.so')!r}\n"
            "print(b.build())")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "left out" in r.stdout and r.stdout.split()[-1] == kbuild.LIB
    assert not (tmp_path / "_kt_ops.so").exists()


def test_the_module_is_built_anew_for_another_torch(lib, tmp_path, monkeypatch):
    assert kbuild._module_is_for(kbuild._module_for())
    monkeypatch.setattr(kbuild, "MODULE_STAMP", str(tmp_path / "stamp"))
    assert not kbuild._module_is_for(kbuild._module_for())  # built by nobody knows what
    (tmp_path / "stamp").write_text(kbuild._module_for())
    assert kbuild._module_is_for(kbuild._module_for())
    monkeypatch.setattr(torch, "__version__", "another")
    assert not kbuild._module_is_for(kbuild._module_for())
