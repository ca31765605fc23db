"""Activations in 8-bit floating point and the linear layer on them, on the GPU."""
import pytest
import torch

from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops

import ops_reference
import train_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_mlp_gemms_gb300 import build
    build.build()
    kt_ops.load()


def quantize(x, K, act=kt_mlp.KT_ACT_NONE, pad=0):
    M = x.shape[0]
    q = torch.full((M, K + pad), 1, dtype=torch.uint8, device="cuda").view(E4)
    scale = torch.full((M, -(-K // 128)), -1.0, device="cuda")
    kt_ops.kt_quantize_fp8(x, q[:, :K], scale, act)
    assert (q.view(torch.uint8)[:, K:] == 1).all()
    return q[:, :K], scale


def same(q, want):
    return torch.equal(q.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,pad", [(1, 1, 0), (1, 128, 0), (3, 16, 0), (5, 37, 3), (9, 640, 0), (729, 1152, 0), (33, 1288, 8), (8, 2048, 16),
                                     (7, 4304, 0), (5, 10241, 0), (4000, 72, 0), (300, 129, 1)])
def test_the_numbers_are_the_nearest(M, K, pad, dtype):
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn(M, K + pad, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))).to(DT[dtype]).cuda()[:, :K]
    q, scale = quantize(x, K, pad=pad)
    qx, sx = ref.e4m3(x, 128)
    assert torch.equal(scale, sx) and same(q, qx)


def test_zeros_subnormals_and_bad_runs():
    dt, K = torch.bfloat16, 512
    x = torch.zeros(6, K)
    x[1, 5], x[1, 300] = 1e-37, -2.0 ** -99
    x[2] = torch.exp2(torch.linspace(-40, 20, K))
    x[3], x[3, 200] = 1.0, float("nan")
    x[4], x[4, 511] = 1.0, float("-inf")
    x[5] = torch.finfo(dt).max
    x = x.to(dt).cuda()
    q, scale = quantize(x, K)
    qx, sx = ref.e4m3(x, 128)
    assert torch.equal(scale.nan_to_num(-7.0), sx.nan_to_num(-7.0))
    assert scale[1, 0] == 0 and scale[1, 2] > 0 and scale[3, 1].isnan() and scale[4, 3].isinf() and scale[4, :3].isfinite().all()
    fine = sx.isfinite().repeat_interleave(128, 1)
    assert torch.equal(q.view(torch.uint8)[fine], qx.view(torch.uint8)[fine])
    assert (q[5].float() == 448).all()


ACTS = {"geglu": kt_mlp.KT_ACT_GEGLU, "gelu_erf": kt_mlp.KT_ACT_GELU_ERF, "gelu_tanh": kt_mlp.KT_ACT_GELU_TANH,
        "gelu_sigmoid": kt_mlp.KT_ACT_GELU_SIGMOID, "silu": kt_mlp.KT_ACT_SILU}


@pytest.mark.parametrize("name", sorted(ACTS))
@pytest.mark.parametrize("M,K", [(5, 72), (33, 1280), (9, 101)])
def test_activations_as_they_are_quantised(name, M, K):
    """The activation is good to 2e-5 (the library's tested bound), so a value may be off by that and by half a step
    of e4m3: 2^-4 of the value, 2^-10 scales below e4m3's normal numbers."""
    g = torch.Generator().manual_seed(K)
    x = (2 * torch.randn(M, 2 * K if name == "geglu" else K, generator=g)).to(torch.bfloat16).cuda()
    q, scale = quantize(x, K, ACTS[name])
    v = ops_reference.act(x.double(), name)
    most = torch.nn.functional.pad(v, (0, -K % 128)).view(M, -1, 128).abs().amax(-1)
    assert ((scale.double() * 448 - most).abs() <= 2.1e-5 * most).all()
    s = scale.double().repeat_interleave(128, 1)[:, :K]
    assert ((q.double() * s - v).abs() <= torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * s) * 1.0001 + 4.2e-5 * v.abs() + 1e-37).all()


def operands(g, M, N, K, dt, bias, pad=0):
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    q, sx = ref.e4m3(x, 128)
    w = torch.randn(N, K + pad, generator=g).mul(60).clamp(-448, 448).to(E4)[:, :K]
    sw = torch.exp(torch.randn(-(-N // 128), -(-K // 128), generator=g)) * (0.02 / K ** 0.5)
    b = torch.randn(N, generator=g).to(dt).cuda() if bias else None
    wide = torch.empty(M, K + pad, dtype=E4)
    wide[:, :K] = q
    big = torch.empty(N, K + pad, dtype=E4)
    big[:, :K] = w
    return wide.cuda()[:, :K], sx.cuda(), big.cuda()[:, :K], sw.cuda(), b


def near(y, q, sx, w, sw, b):
    yx, tol = ref.linear_fp8(q, sx, w, sw, b)
    tol = ref.rounded(yx, tol, y.dtype)
    bad = ~((y.double() - yx).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), y[bad][0].item(), yx[bad][0].item(), tol[bad][0].item())


# few tokens (one, two and four column groups; alone and shared by clusters), one tile and many, ragged everywhere
SHAPES = [(1, 8, 16), (1, 128, 128), (3, 40, 48), (4, 10240, 1280), (16, 1280, 5120), (17, 264, 8192), (33, 1000, 640), (64, 520, 4112),
          (64, 30000, 144), (65, 8, 16), (100, 136, 272), (128, 256, 128), (129, 256, 2048), (300, 4304, 1152), (729, 1152, 4304), (1000, 520, 80),
          (2500, 2560, 1168), (5000, 1032, 1024), (140, 9728, 640), (700, 5000, 3088)]


@pytest.mark.parametrize("dtype,bias", [("f16", True), ("bf16", False)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(M, N, K, dtype, bias):
    g = torch.Generator().manual_seed(M * 7 + N * 3 + K)
    dt = DT[dtype]
    args = operands(g, M, N, K, dt, bias, pad=16)
    whole = torch.full((M, N + 8), float("nan"), dtype=dt, device="cuda")
    kt_ops.kt_linear_fp8(*args, whole[:, :N])
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    near(whole[:, :N], *args)
    assert whole[:, N:].isnan().all()
    again = torch.empty_like(whole)[:, :N]
    kt_ops.kt_linear_fp8(*args, again)
    assert torch.equal(again, whole[:, :N])


@pytest.mark.parametrize("M", [4, 100, 600])
def test_sums_that_cancel_within_a_run_are_exact(M):
    """Products of whole numbers whose partial sums pass 2^17 and come back to small integers: not one unit is lost in a
    run's fp32 sum; the runs' scales are powers of two apart."""
    g = torch.Generator().manual_seed(M)
    N, K = 136, 384
    q = torch.randint(-15, 16, (M, K), generator=g).float()
    half = torch.randint(-15, 16, (N, 64), generator=g).float()
    w = torch.cat([torch.cat([half, -half], 1)] * 3, 1)
    q[:, 64:128], q[:, 192:256], q[:, 320:] = q[:, :64], q[:, 128:192], q[:, 256:320]
    q[:, [127, 255]] = torch.randint(-15, 16, (M, 2), generator=g).float()
    q *= 16.0
    assert (q.abs() <= 240).all()  # 4 significant bits: e4m3 holds them
    qe, we = q.to(E4), w.to(E4)
    assert torch.equal(qe.float(), q) and torch.equal(we.float(), w)
    sx, sw = torch.full((M, 3), 2.0 ** -4), torch.tensor([[1.0, 2.0, 0.5]] * 2)
    y = torch.empty(M, N, dtype=torch.float16, device="cuda")
    kt_ops.kt_linear_fp8(qe.cuda(), sx.cuda(), we.cuda(), sw.cuda(), None, y)
    exact = sum((q[:, k:k + 128].double() @ w[:, k:k + 128].double().t()) / 16 * s for k, s in ((0, 1.0), (128, 2.0), (256, 0.5)))
    assert exact.abs().max() <= 2048 and exact.unique().numel() > 10
    assert torch.equal(y.cpu().double(), exact)


@pytest.mark.parametrize("M", [5, 200])
def test_a_bad_token_is_its_own(M):
    g = torch.Generator().manual_seed(M)
    N, K = 264, 400
    q, sx, w, sw, _ = operands(g, M, N, K, torch.float16, False)
    y = torch.empty(M, N, dtype=torch.float16, device="cuda")
    kt_ops.kt_linear_fp8(q, sx, w, sw, None, y)
    want = y.clone()
    sx[3, 1] = float("nan")
    kt_ops.kt_linear_fp8(q, sx, w, sw, None, y)
    assert y[3].isnan().all()
    others = torch.arange(M, device="cuda") != 3
    assert torch.equal(y[others], want[others])


def test_no_tokens():
    e = lambda n, d: torch.empty(0, n, dtype=d, device="cuda")  # noqa: E731
    kt_ops.kt_quantize_fp8(e(64, torch.float16), e(64, E4), e(1, torch.float32))
    kt_ops.kt_linear_fp8(e(64, E4), e(1, torch.float32), torch.zeros(8, 64, dtype=torch.uint8, device="cuda").view(E4),
                         torch.zeros(1, 1, device="cuda"), None, e(8, torch.float16))
    torch.cuda.synchronize()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("M,N,K", [(4, 1280, 640), (64, 640, 4096), (300, 520, 272), (729, 4304, 640)])
def test_new_values_in_the_same_buffers_are_read(M, N, K, captured):
    """Tokens quantised into the same buffers right before each product: every step's result is that of the step alone."""
    g = torch.Generator().manual_seed(M + K)
    steps = 10
    x = torch.randn(steps, M, K, generator=g).to(torch.bfloat16).cuda()
    _, _, w, sw, _ = operands(g, 1, N, K, torch.bfloat16, False)

    def step(i, q, s, y):
        kt_ops.kt_quantize_fp8(x[i], q, s)
        kt_ops.kt_linear_fp8(q, s, w, sw, None, y)

    def buffers():
        return torch.zeros(M, K, dtype=torch.uint8, device="cuda").view(E4), torch.zeros(M, -(-K // 128), device="cuda")

    alone = torch.full((steps, M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i in range(steps):
        q, s = buffers()
        step(i, q, s, alone[i])
        torch.cuda.synchronize()
        near(alone[i], q, s, w, sw, None)
    q, s = buffers()
    got = torch.full_like(alone, float("nan"))
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(steps):
                step(i, q, s, got[i])
        graph.replay()
        torch.cuda.synchronize()
        got.fill_(float("nan"))
        graph.replay()
    else:
        for i in range(steps):
            step(i, q, s, got[i])
    torch.cuda.synchronize()
    for i in range(steps):
        assert torch.equal(got[i], alone[i]), i


@pytest.mark.parametrize("M,N,K", [(4, 1280, 640), (64, 640, 4096), (100, 136, 272), (140, 9728, 640), (3000, 2560, 640), (100, 256, 8192)])
def test_a_wait_that_runs_out_is_reported_and_shows(M, N, K):
    g = torch.Generator().manual_seed(M)
    args = operands(g, M, N, K, torch.float16, False)
    want = torch.empty(M, N, dtype=torch.float16, device="cuda")
    kt_ops.kt_linear_fp8(*args, want)
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    whole = torch.full((M, N + 8), 7.0, dtype=torch.float16, device="cuda")
    got = whole[:, :N]
    kt_ops.kt_matmul_debug_stall(True, 20000)
    try:
        kt_ops.kt_linear_fp8(*args, got)
        assert kt_ops.kt_matmul_status() == kt_mlp.KT_ERR_TIMEOUT
    finally:
        kt_ops.kt_matmul_debug_stall(False)
    bad = got.isnan()
    assert bad[0, 0] and (bad | (got == want)).all()
    assert (whole[:, N:] == 7).all()
    kt_ops.kt_linear_fp8(*args, got)
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    assert torch.equal(got, want)
