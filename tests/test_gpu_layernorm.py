"""Layer norm and its gradients on the GPU against the 64-bit formulas (ops_reference), element
by element within bounds that count roundings."""
import pytest
import torch

from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops

import ops_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_mlp_gemms_gb300 import build
    build.build()
    kt_ops.load()


def rows(M, D, pad, dtype, seed, offset=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, D + pad, generator=g) * (0.25 + 4 * torch.rand(M, 1, generator=g)) + offset * torch.randn(M, 1, generator=g)
    return x.to(dtype).cuda()[:, :D]


def affine(D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda(), (0.1 * torch.randn(D, generator=g)).to(dtype).cuda()


def within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} elements, first {bad.nonzero()[0].tolist()}: " \
                          f"{got[bad][0].item()} for {want[bad][0].item()} +- {tol.expand_as(want)[bad][0].item()}"


# every team shape (1 to 16 warps, 1 to 5 slots), odd lengths and pitches, one row and many
SHAPES = [(1, 1, 0), (3, 8, 0), (5, 33, 0), (9, 256, 0), (8, 264, 8), (33, 643, 6), (64, 640, 0), (129, 1000, 0), (729, 1152, 0),
          (37, 1280, 8), (17, 1281, 0), (16, 1536, 0), (11, 2048, 0), (7, 2056, 0), (5, 4096, 16), (6, 4099, 3), (4, 6144, 0),
          (3, 8192, 0), (4, 8200, 0), (3, 12288, 0), (5, 16384, 0), (2, 16383, 1), (5000, 40, 0), (3001, 96, 5),
          # many rows per team: the backward pass's rows come through the ring
          (3800, 1280, 0), (9000, 640, 8), (4001, 1000, 0), (2500, 2048, 0), (1500, 4096, 0), (1000, 6144, 0), (700, 8192, 0)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,D,pad", SHAPES)
def test_forward_and_backward(M, D, pad, dtype):
    dt = DT[dtype]
    x = rows(M, D, pad, dt, 7 * M + D)
    gamma, beta = affine(D, dt, D)
    y = torch.full((M, D + pad), float("nan"), dtype=dt, device="cuda")[:, :D]
    mean, rstd = torch.full((M,), float("nan"), device="cuda"), torch.full((M,), float("nan"), device="cuda")
    kt_ops.kt_layernorm_forward(x, gamma, beta, EPS, y, mean, rstd)
    yx, mx, rx = ref.layernorm(x, gamma, beta, EPS)
    ty, tm, tr = ref.layernorm_bounds(x, gamma, beta, yx, rx, dt)
    within(mean, mx, tm, "mean")
    within(rstd, rx, tr, "rstd")
    within(y, yx, ty, "y")

    dy = rows(M, D, pad, dt, 11 * M + D, 0.3)
    dx = torch.full((M, D + pad), float("nan"), dtype=dt, device="cuda")[:, :D]
    dgamma, dbeta = torch.full((D,), float("nan"), device="cuda"), torch.full((D,), float("nan"), device="cuda")
    ws = kt_ops.layernorm_backward_workspace(M, D)
    ws.fill_(255)  # its content does not matter
    kt_ops.kt_layernorm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws)
    dxx, dgx, dbx = ref.layernorm_backward(dy, x, gamma, mean, rstd)
    tx, tg, tb = ref.layernorm_backward_bounds(dy, x, gamma, mean, rstd, dxx, dt)
    within(dx, dxx, tx, "dx")
    within(dgamma, dgx, tg, "dgamma")
    within(dbeta, dbx, tb, "dbeta")


@pytest.mark.parametrize("M,D", [(65, 1280), (9, 77)])
def test_without_affine_statistics_or_sums(M, D):
    x, dy = rows(M, D, 0, torch.bfloat16, 1), rows(M, D, 0, torch.bfloat16, 2)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    kt_ops.kt_layernorm_forward(x, None, None, EPS, y)
    yx, mx, rx = ref.layernorm(x, None, None, EPS)
    within(y, yx, ref.layernorm_bounds(x, None, None, yx, rx, x.dtype)[0], "y")
    mean, rstd = mx.float(), rx.float()
    kt_ops.kt_layernorm_backward(dy, x, None, mean, rstd, dx)
    dxx = ref.layernorm_backward(dy, x, None, mean, rstd)[0]
    within(dx, dxx, ref.layernorm_backward_bounds(dy, x, None, mean, rstd, dxx, x.dtype)[0], "dx")


def test_no_rows_and_constant_rows():
    D = 72
    gamma, beta = affine(D, torch.float16, 3)
    empty = torch.empty(0, D, dtype=torch.float16, device="cuda")
    none = torch.empty(0, device="cuda")
    kt_ops.kt_layernorm_forward(empty, gamma, beta, EPS, empty, none, none)
    dgamma, dbeta = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    kt_ops.kt_layernorm_backward(empty, empty, gamma, none, none, empty, dgamma, dbeta, kt_ops.layernorm_backward_workspace(0, D))
    assert (dgamma == 0).all() and (dbeta == 0).all()
    x = torch.full((3, D), 1234.0, dtype=torch.float16, device="cuda")  # no spread at all: y is beta, exactly
    y, mean, rstd = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    kt_ops.kt_layernorm_forward(x, gamma, beta, EPS, y, mean, rstd)
    assert (y == beta).all() and (mean == 1234.0).all()
    assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=4e-7)


def test_a_row_far_from_zero_keeps_its_digits():
    g = torch.Generator().manual_seed(5)
    x = (30000.0 + 16.0 * torch.randint(-3, 4, (5, 1280), generator=g)).to(torch.float16).cuda()
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    kt_ops.kt_layernorm_forward(x, None, None, EPS, y, mean, rstd)
    yx, mx, rx = ref.layernorm(x, None, None, EPS)
    ty, tm, tr = ref.layernorm_bounds(x, None, None, yx, rx, x.dtype)
    within(mean, mx, tm, "mean")
    within(rstd, rx, tr, "rstd")
    within(y, yx, ty, "y")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_value_stays_in_its_row(value):
    x = rows(9, 1280, 0, torch.bfloat16, 6)
    clean, y = torch.empty_like(x), torch.empty_like(x)
    kt_ops.kt_layernorm_forward(x, None, None, EPS, clean)
    x = x.clone()
    x[4, 700] = value
    kt_ops.kt_layernorm_forward(x, None, None, EPS, y)
    assert y[4].isnan().all()
    keep = [r for r in range(9) if r != 4]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("D", [1280, 2001])
def test_in_place_and_from_run_to_run(D):
    M = 3000
    x, dy = rows(M, D, 0, torch.bfloat16, 8), rows(M, D, 0, torch.bfloat16, 9)
    gamma, beta = affine(D, torch.bfloat16, 10)
    y, mean, rstd = torch.empty_like(x), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    kt_ops.kt_layernorm_forward(x, gamma, beta, EPS, y, mean, rstd)
    z = x.clone()
    kt_ops.kt_layernorm_forward(z, gamma, beta, EPS, z)
    assert torch.equal(z, y)
    ws = kt_ops.layernorm_backward_workspace(M, D)
    outs = []
    for where in ("new", "new", "dy", "x"):
        a, b = dy.clone(), x.clone()
        dx = {"new": torch.empty_like(x), "dy": a, "x": b}[where]
        dgamma, dbeta = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        kt_ops.kt_layernorm_backward(a, b, gamma, mean, rstd, dx, dgamma, dbeta, ws)
        outs.append((dx, dgamma, dbeta))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


def test_gradients_against_differences_of_the_kernel_inputs():
    """dgamma and dbeta (fp32) against central differences of the 64-bit loss; its quotients are
    good to 1e-7 of the terms' sum (h = 1e-4), the kernel's sums to their bound."""
    M, D, h = 13, 24, 1e-4
    x, dy = rows(M, D, 0, torch.float16, 12, 0.5), rows(M, D, 0, torch.float16, 13, 0.5)
    gamma, beta = affine(D, torch.float16, 14)
    _, mx, rx = ref.layernorm(x, gamma, beta, EPS)
    mean, rstd, dx = mx.float(), rx.float(), torch.empty_like(x)
    dgamma, dbeta = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    kt_ops.kt_layernorm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, kt_ops.layernorm_backward_workspace(M, D))
    args = [x.double(), gamma.double(), beta.double()]

    def loss(a):
        return (ref.layernorm(*a, EPS)[0] * dy.double()).sum()

    dxx, _, _ = ref.layernorm_backward(dy, x, gamma, mean, rstd)
    tols = ref.layernorm_backward_bounds(dy, x, gamma, mean, rstd, dxx, x.dtype)
    for which, grad, tol in ((0, dx, tols[0]), (1, dgamma, tols[1]), (2, dbeta, tols[2])):
        for i in range(0, args[which].numel(), 7):
            quotients = []
            for sign in (1, -1):
                a = [t.clone() for t in args]
                a[which].view(-1)[i] += sign * h
                quotients.append(loss(a))
            d = (quotients[0] - quotients[1]) / (2 * h)
            assert abs(d - grad.reshape(-1)[i].double()) <= tol.reshape(-1)[i] + 1e-6


def test_graph_and_another_stream():
    M, D = 300, 1152
    x, dy = rows(M, D, 0, torch.float16, 15), rows(M, D, 0, torch.float16, 16)
    gamma, beta = affine(D, torch.float16, 17)
    ws = kt_ops.layernorm_backward_workspace(M, D)

    def step(out):
        kt_ops.kt_layernorm_forward(x, gamma, beta, EPS, out["y"], out["mean"], out["rstd"])
        kt_ops.kt_layernorm_backward(dy, x, gamma, out["mean"], out["rstd"], out["dx"], out["dgamma"], out["dbeta"], ws)

    def outputs():
        f = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
        return {"y": f(M, D).half(), "mean": f(M), "rstd": f(M), "dx": f(M, D).half(), "dgamma": f(D), "dbeta": f(D)}

    eager, captured, side = outputs(), outputs(), outputs()
    step(eager)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for k in eager:
        assert torch.equal(eager[k], captured[k]) and torch.equal(eager[k], side[k]), k
    # new values in the captured tensors: replays read them
    x.copy_(rows(M, D, 0, torch.float16, 18))
    graph.replay()
    step(eager)
    torch.cuda.synchronize()
    assert all(torch.equal(eager[k], captured[k]) for k in eager)


def test_refusals_with_tensors():
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    f = torch.zeros(4, device="cuda")
    for call in (lambda: kt_ops.kt_layernorm_forward(x, None, None, EPS, x.cpu()),
                 lambda: kt_ops.kt_layernorm_forward(x, None, None, -1.0, x),
                 lambda: kt_ops.kt_layernorm_backward(x, x, None, f, f, x, torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")),
                 lambda: kt_ops.kt_layernorm_backward(x, x, None, f, f, x, f, f)):
        with pytest.raises(kt_mlp.KtError) as e:
            call()
        assert e.value.status == kt_mlp.KT_ERR_INVALID


@pytest.mark.parametrize("M,D,pad", [(1000, 2051, 0), (1300, 1281, 2), (700, 4099, 3), (500, 8191, 0), (400, 8200, 1), (5000, 257, 0), (4000, 770, 5)])
def test_several_rows_per_team_at_any_pitch(M, D, pad):
    test_forward_and_backward(M, D, pad, "f16")


@pytest.mark.parametrize("M,D", [(729, 1152), (100, 643), (3800, 1280)])
def test_new_values_in_the_same_workspace_are_read(M, D):
    """Backward passes of changing inputs right behind one another through one workspace: each step's
    sums are those of the step alone, bit for bit."""
    steps = 10
    gamma, _ = affine(D, torch.float16, 20)
    inputs = []
    for i in range(steps):
        x, dy = rows(M, D, 0, torch.float16, 21 + i), rows(M, D, 0, torch.float16, 51 + i, 0.3)
        _, mean, rstd = ref.layernorm(x, None, None, EPS)
        inputs.append((dy, x, gamma, mean.float(), rstd.float()))
    ws = kt_ops.layernorm_backward_workspace(M, D)

    def step(i):
        out = torch.full((M, D), float("nan"), dtype=torch.float16, device="cuda"), *(torch.full((2, D), float("nan"), device="cuda"))
        kt_ops.kt_layernorm_backward(*inputs[i], *out, ws)
        return out

    alone = []
    for i in range(steps):
        alone.append(step(i))
        torch.cuda.synchronize()
    again = [step(i) for i in range(steps)]
    torch.cuda.synchronize()
    for a, b in zip(alone, again):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("column", [0, 7, -1])
@pytest.mark.parametrize("dtype,outlier", [("f16", 3e3), ("f16", -3e4), ("bf16", 6e4), ("bf16", 1e6)])
@pytest.mark.parametrize("D", [40, 643, 1280, 4096, 4099, 16384])
def test_one_value_far_from_the_others(D, dtype, outlier, column):
    """One large value in a row, the first one too: the mean and the other elements keep their digits."""
    dt, M = DT[dtype], 7
    x = rows(M, D, 0, dt, D, 0.5)
    x[:, column] = outlier
    gamma, beta = affine(D, dt, D + 1)
    y, mean, rstd = torch.empty_like(x), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    kt_ops.kt_layernorm_forward(x, gamma, beta, EPS, y, mean, rstd)
    yx, mx, rx = ref.layernorm(x, gamma, beta, EPS)
    ty, tm, tr = ref.layernorm_bounds_about_the_mean(x, gamma, beta, yx, mx, rx, dt)
    within(mean, mx, tm, "mean")
    within(rstd, rx, tr, "rstd")
    within(y, yx, ty, "y")


@pytest.mark.parametrize("value", [1e-30, 1e30, 2e36, 3e38])
def test_equal_values_of_any_size(value):
    """Rows without spread whose sum may be beyond fp32: y is beta and the mean the value, exactly."""
    for D in (72, 643, 1152, 16384):
        gamma, beta = affine(D, torch.bfloat16, D)
        x = torch.full((3, D), value, dtype=torch.bfloat16, device="cuda")
        y, mean, rstd = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
        kt_ops.kt_layernorm_forward(x, gamma, beta, EPS, y, mean, rstd)
        assert (y == beta).all() and (mean == x[:, 0].float()).all()
        assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=4e-7)


@pytest.mark.parametrize("D", [5, 72, 643, 1152, 1280, 2051, 4096, 4099, 16383])
@pytest.mark.parametrize("value,eps", [(2e36, 1e-5), (1e33, 1e-20)])
def test_gradients_of_large_equal_values(D, value, eps):
    """mean * rstd beyond fp32: xhat is 0 throughout and dx finite, whatever the row's length leaves
    over of a lane's slots."""
    M = 600
    x = torch.full((M, D), value, dtype=torch.bfloat16, device="cuda")
    dy = rows(M, D, 0, torch.bfloat16, D, 0.3)
    gamma, _ = affine(D, torch.bfloat16, D)
    mean, rstd = x[:, 0].float(), torch.full((M,), eps ** -0.5, device="cuda")
    dx = torch.full((M, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgamma, dbeta = torch.full((D,), float("nan"), device="cuda"), torch.full((D,), float("nan"), device="cuda")
    kt_ops.kt_layernorm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, kt_ops.layernorm_backward_workspace(M, D))
    dxx, dgx, dbx = ref.layernorm_backward(dy, x, gamma, mean, rstd)
    tx, tg, tb = ref.layernorm_backward_bounds(dy, x, gamma, mean, rstd, dxx, x.dtype)
    within(dx, dxx, tx, "dx")
    within(dgamma, dgx, tg, "dgamma")
    within(dbeta, dbx, tb, "dbeta")
