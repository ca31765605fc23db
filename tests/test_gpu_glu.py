"""The gated up projection and the linear layer, forward and backward, on the GPU against their 64-bit forms."""
import pytest
import torch

from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops

import train_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTS = {"gelu_erf": kt_mlp.KT_ACT_GELU_ERF, "gelu_tanh": kt_mlp.KT_ACT_GELU_TANH, "gelu_sigmoid": kt_mlp.KT_ACT_GELU_SIGMOID,
        "silu": kt_mlp.KT_ACT_SILU, "none": kt_mlp.KT_ACT_NONE}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_mlp_gemms_gb300 import build
    build.build()
    kt_ops.load()


def randn(g, *shape, dtype, std=1.0, pad=0):
    """A matrix whose rows are pad elements apart from one another."""
    t = (std * torch.randn(*shape[:-1], shape[-1] + pad, generator=g)).to(dtype).cuda()
    return t[..., :shape[-1]]


def nans(M, N, dtype, pad=0):
    """The whole buffer and the matrix in it."""
    whole = torch.full((M, N + pad), float("nan"), dtype=dtype, device="cuda")
    return whole, whole[:, :N]


def near(got, want, tol):
    # what is past the type's largest number and half a step rounds to infinity (300 * 300 = 90000 in float16)
    past = want.abs() - tol > torch.finfo(got.dtype).max * (1 + ref.half(got.dtype))
    bad = ~torch.where(past, got.double() == torch.copysign(torch.full_like(want, float("inf")), want), (got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item(), tol[bad][0].item())


# one tile and many, ragged in every direction; single CTAs, pairs; one token to several row blocks per pair
SHAPES = [(1, 8, 8), (1, 64, 640), (3, 72, 200), (64, 640, 1000), (129, 136, 72), (300, 256, 520), (729, 1152, 4304), (2500, 640, 328),
          (5000, 264, 2560)]


@pytest.mark.parametrize("dtype,bias", [("f16", True), ("bf16", False)])
@pytest.mark.parametrize("M,D,F", SHAPES)
def test_gated_projection(M, D, F, dtype, bias):
    g = torch.Generator().manual_seed(M + D + F)
    dt, name = DT[dtype], sorted(ACTS)[(M + D) % len(ACTS)]
    x, w = randn(g, M, D, dtype=dt, pad=8), randn(g, 2 * F, D, dtype=dt, std=D ** -0.5)
    b = randn(g, 2 * F, dtype=dt, std=0.2) if bias else None
    hs, h = nans(M, F, dt, 16)
    ps, p = nans(M, 2 * F, dt, 8)
    kt_ops.kt_glu_forward(x, w, b, h, p, ACTS[name])
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    hx, th, px, tp = ref.glu(x, w, b, name, dt)
    near(p, px, tp)
    near(h, hx, th)
    assert hs[:, F:].isnan().all() and ps[:, 2 * F:].isnan().all()
    alone = torch.empty_like(h)
    kt_ops.kt_glu_forward(x, w, b, alone, None, ACTS[name])  # the same h without p
    assert torch.equal(alone, h)


@pytest.mark.parametrize("name", sorted(ACTS))
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gates_of_every_size(name, dtype):
    """W the identity: gates from far below to far above, through both passes; nothing that is finite turns into NaN."""
    dt, F = DT[dtype], 64
    span = torch.cat([torch.linspace(-12, 12, 40), torch.tensor([-300.0, -88.0, -40.0, 40.0, 88.0, 300.0, 0.0, -0.0]),
                      torch.linspace(-1, 1, 16)]).to(dt)
    value = torch.linspace(-2, 2, F).to(dt)
    x = torch.stack([torch.cat([value, span]), torch.cat([-value, span.flip(0)])]).cuda()
    w = torch.eye(2 * F, dtype=dt).cuda()
    h, p = torch.empty(2, F, dtype=dt, device="cuda"), torch.empty(2, 2 * F, dtype=dt, device="cuda")
    kt_ops.kt_glu_forward(x, w, None, h, p, ACTS[name])
    assert torch.equal(p, x)
    hx, th, _, _ = ref.glu(x, w, None, name, dt)
    near(h, hx, th)
    dh = torch.ones_like(h)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(2 * F, device="cuda")
    kt_ops.kt_glu_backward(dh, p, x, w, dx, dw, db, ACTS[name], kt_ops.glu_backward_workspace(2, 2 * F, F))
    dxx, tx, dwx, tw, dbx, tb = ref.glu_backward(dh, p, x, w, name, dt)
    near(dx, dxx, tx)
    near(dw, dwx, tw)
    near(db, dbx, tb)


@pytest.mark.parametrize("dtype,bias", [("f16", False), ("bf16", True)])
@pytest.mark.parametrize("M,D,F", SHAPES)
def test_gated_gradients(M, D, F, dtype, bias):
    g = torch.Generator().manual_seed(M * 3 + D + F)
    dt, name = DT[dtype], sorted(ACTS)[(M + F) % len(ACTS)]
    x, w = randn(g, M, D, dtype=dt, pad=16), randn(g, 2 * F, D, dtype=dt, std=D ** -0.5)
    p, dh = randn(g, M, 2 * F, dtype=dt, pad=8), randn(g, M, F, dtype=dt, std=0.5, pad=24)
    dxs, dx = nans(M, D, dt, 8)
    dw = torch.full((2 * F, D), float("nan"), dtype=dt, device="cuda")
    db = torch.full((2 * F,), float("nan"), device="cuda") if bias else None
    ws = kt_ops.glu_backward_workspace(M, D, F)
    ws.fill_(255)  # its content is irrelevant: NaN as 16-bit and as 32-bit numbers
    kt_ops.kt_glu_backward(dh, p, x, w, dx, dw, db, ACTS[name], ws)
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    dxx, tx, dwx, tw, dbx, tb = ref.glu_backward(dh, p, x, w, name, dt)
    near(dx, dxx, tx)
    near(dw, dwx, tw)
    if bias:
        near(db, dbx, tb)
    assert dxs[:, D:].isnan().all()
    # the same bits again; and each gradient alone, whose sums may be shared out in another way
    again = [torch.empty_like(dx), torch.empty_like(dw)]
    kt_ops.kt_glu_backward(dh, p, x, w, *again, None, ACTS[name], ws)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    kt_ops.kt_glu_backward(dh, p, x, w, again[0].fill_(float("nan")), None, None, ACTS[name], ws)
    near(again[0], dxx, tx)
    kt_ops.kt_glu_backward(dh, p, x, w, None, again[1].fill_(float("nan")), None, ACTS[name], ws)
    near(again[1], dwx, tw)


# also long sums of few tiles, which a cluster shares
LINEAR = [(1, 8, 8), (2, 640, 2560), (17, 72, 5120), (100, 128, 8192), (331, 640, 2560), (129, 1000, 72), (729, 1152, 4304),
          (2048, 64, 64), (16384, 64, 136), (4000, 2560, 640), (700, 5000, 1288)]


@pytest.mark.parametrize("dtype,bias", [("f16", True), ("bf16", False)])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_layer(M, N, K, dtype, bias):
    g = torch.Generator().manual_seed(M + 5 * N + K)
    dt = DT[dtype]
    x, w, dy = randn(g, M, K, dtype=dt, pad=8), randn(g, N, K, dtype=dt, std=K ** -0.5), randn(g, M, N, dtype=dt, std=0.25, pad=8)
    b = randn(g, N, dtype=dt) if bias else None
    ys, y = nans(M, N, dt, 8)
    kt_ops.kt_linear_forward(x, w, b, y)
    yx, ty = ref.product(x.double(), w.double(), b)
    near(y, yx, ref.rounded(yx, ty, dt))
    dxs, dx = nans(M, K, dt, 16)
    dw = torch.full((N, K), float("nan"), dtype=dt, device="cuda")
    db = torch.full((N,), float("nan"), device="cuda") if bias else None
    kt_ops.kt_linear_backward(dy, x, w, dx, dw, db, kt_ops.linear_backward_workspace(M, N, K))
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    dxx, tx, dwx, tw, dbx, tb = ref.linear_backward(dy, x, w, dt)
    near(dx, dxx, tx)
    near(dw, dwx, tw)
    if bias:
        near(db, dbx, tb)
    assert ys[:, N:].isnan().all() and dxs[:, K:].isnan().all()


def test_no_tokens():
    D, F = 64, 72
    e = lambda n: torch.empty(0, n, dtype=torch.float16, device="cuda")  # noqa: E731
    w = torch.ones(2 * F, D, dtype=torch.float16, device="cuda")
    kt_ops.kt_glu_forward(e(D), w, None, e(F), e(2 * F), kt_mlp.KT_ACT_SILU)
    dw, db = torch.ones_like(w), torch.ones(2 * F, device="cuda")
    kt_ops.kt_glu_backward(e(F), e(2 * F), e(D), w, e(D), dw, db, kt_mlp.KT_ACT_SILU, kt_ops.glu_backward_workspace(0, D, F))
    assert not dw.any() and not db.any()
    kt_ops.kt_linear_forward(e(D), w, None, e(2 * F))
    dw, db = torch.ones_like(w), torch.ones(2 * F, device="cuda")
    kt_ops.kt_linear_backward(e(2 * F), e(D), w, e(D), dw, db, kt_ops.linear_backward_workspace(0, 2 * F, D))
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_is_its_own(bad):
    """A token with a NaN or an infinity spoils its own rows and the sums over the tokens, and no other row: not even where
    the rows past the last token are filled up."""
    g = torch.Generator().manual_seed(2)
    M, D, F, dt = 200, 72, 136, torch.bfloat16
    x, w = randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=0.1)
    x[77, 5] = bad
    h, p = torch.empty(M, F, dtype=dt, device="cuda"), torch.empty(M, 2 * F, dtype=dt, device="cuda")
    kt_ops.kt_glu_forward(x, w, None, h, p, kt_mlp.KT_ACT_SILU)
    others = torch.arange(M, device="cuda") != 77
    assert not p[77].isfinite().any() and p[others].isfinite().all() and h[others].isfinite().all()
    dh = randn(g, M, F, dtype=dt)
    dh[77, 3] = bad
    p[77] = 1.0
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(2 * F, device="cuda")
    kt_ops.kt_glu_backward(dh, p, x, w, dx, dw, db, kt_mlp.KT_ACT_SILU, kt_ops.glu_backward_workspace(M, D, F))
    assert not dx[77].isfinite().any() and dx[others].isfinite().all()
    clean = torch.arange(2 * F, device="cuda") % F != 3
    assert not db[~clean].isfinite().any() and db[clean].isfinite().all()
    assert not dw[~clean].isfinite().any()
    assert dw[clean][:, torch.arange(D, device="cuda") != 5].isfinite().all()


def step(x, w, b, dh, out, name=kt_mlp.KT_ACT_GELU_ERF):
    h, p, dx, dw, db, ws = out
    kt_ops.kt_glu_forward(x, w, b, h, p, name)
    kt_ops.kt_glu_backward(dh, p, x, w, dx, dw, db, name, ws)


def outputs(M, D, F, dt):
    whole = [torch.full(s, float("nan"), dtype=dt, device="cuda") for s in ((M, F), (M, 2 * F), (M, D), (2 * F, D))]
    return whole + [torch.full((2 * F,), float("nan"), device="cuda"), kt_ops.glu_backward_workspace(M, D, F)]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("M,D,F", [(4, 256, 328), (200, 640, 264), (700, 264, 1000)])
def test_new_values_in_the_same_buffers_are_read(M, D, F, captured):
    """Weights, bias, tokens and gradients written anew right before each step, into the same buffers: every step's
    results are those of the step alone, bit for bit."""
    g = torch.Generator().manual_seed(M)
    dt, steps = torch.bfloat16, 10
    new = [[randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=D ** -0.5), randn(g, 2 * F, dtype=dt), randn(g, M, F, dtype=dt)]
           for _ in range(steps)]
    alone = []
    for n in new:
        out = outputs(M, D, F, dt)
        step(*n, out)
        torch.cuda.synchronize()
        alone.append(out)
    held = [torch.zeros_like(t) for t in new[0]]
    got = [outputs(M, D, F, dt)[:5] for _ in range(steps)]
    ws = kt_ops.glu_backward_workspace(M, D, F)

    def run():
        for n, out in zip(new, got):
            for to, value in zip(held, n):
                to.copy_(value)
            step(*held, out + [ws])

    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graph.replay()
        torch.cuda.synchronize()
        for out in got:
            for t in out:
                t.fill_(float("nan"))
        graph.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    for i in range(steps):
        for a, b in zip(got[i], alone[i]):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    g = torch.Generator().manual_seed(8)
    M, D, F, dt = 500, 328, 520, torch.float16
    args = [[randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=0.05), None, randn(g, M, F, dtype=dt)] for _ in range(2)]
    want = [outputs(M, D, F, dt) for _ in range(2)]
    for a, o in zip(args, want):
        step(*a, o)
    torch.cuda.synchronize()
    got = [outputs(M, D, F, dt) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, o, s in zip(args, got, streams):
            with torch.cuda.stream(s):
                step(*a, o)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a[:5], b[:5]))


@pytest.mark.parametrize("M,N,K", [(100, 136, 272), (1000, 4304, 640), (8000, 2560, 640), (64, 128, 8192)])
def test_a_wait_that_runs_out_is_reported_and_shows(M, N, K):
    """The first block waits, for 20 ms, on a barrier that nobody signals: the status says so, its tiles are NaN and nothing
    is left unwritten, and the next call is right again."""
    g = torch.Generator().manual_seed(M)
    dt = torch.float16
    x, w = randn(g, M, K, dtype=dt), randn(g, N, K, dtype=dt, std=K ** -0.5)
    want = torch.empty(M, N, dtype=dt, device="cuda")
    kt_ops.kt_linear_forward(x, w, None, want)
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    whole = torch.full((M, N + 8), 7.0, dtype=dt, device="cuda")
    got = whole[:, :N]
    kt_ops.kt_matmul_debug_stall(True, 20000)
    try:
        kt_ops.kt_linear_forward(x, w, None, got)
        assert kt_ops.kt_matmul_status() == kt_mlp.KT_ERR_TIMEOUT
    finally:
        kt_ops.kt_matmul_debug_stall(False)
    bad = got.isnan()
    assert bad[0, 0] and (bad | (got == want)).all()
    assert (whole[:, N:] == 7).all()
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    kt_ops.kt_linear_forward(x, w, None, got)
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    assert torch.equal(got, want)


def test_a_gated_wait_that_runs_out_shows():
    g = torch.Generator().manual_seed(1)
    M, D, F, dt = 600, 264, 1000, torch.bfloat16
    x, w = randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=0.05)
    want, got = torch.empty(M, F, dtype=dt, device="cuda"), torch.full((M, F), 7.0, dtype=dt, device="cuda")
    p, q = torch.empty(M, 2 * F, dtype=dt, device="cuda"), torch.full((M, 2 * F), 7.0, dtype=dt, device="cuda")
    kt_ops.kt_glu_forward(x, w, None, want, p, kt_mlp.KT_ACT_SILU)
    kt_ops.kt_matmul_debug_stall(True, 20000)
    try:
        kt_ops.kt_glu_forward(x, w, None, got, q, kt_mlp.KT_ACT_SILU)
        assert kt_ops.kt_matmul_status() == kt_mlp.KT_ERR_TIMEOUT
    finally:
        kt_ops.kt_matmul_debug_stall(False)
    for a, b in ((got, want), (q, p)):
        assert a[0, 0].isnan() and (a.isnan() | (a == b)).all()


def test_offsets_past_32_bits():
    """Rows of a buffer of more than 2^32 elements, far apart: the pitch counts in 64 bits."""
    dt, K, N, M = torch.bfloat16, 64, 64, 5
    pitch = (1 << 30) + 8
    big = torch.empty((M - 1) * pitch + K, dtype=dt, device="cuda")
    x = big.as_strided((M, K), (pitch, 1))
    g = torch.Generator().manual_seed(4)
    x.copy_(torch.randn(M, K, generator=g).to(dt))
    w = randn(g, N, K, dtype=dt, std=0.125)
    y = torch.empty(M, N, dtype=dt, device="cuda")
    kt_ops.kt_linear_forward(x, w, None, y)
    yx, ty = ref.product(x.double(), w.double())
    near(y, yx, ref.rounded(yx, ty, dt))
    dw, db = torch.empty(K, N, dtype=dt, device="cuda"), torch.empty(K, device="cuda")
    kt_ops.kt_linear_backward(x, y, torch.zeros_like(dw), None, dw, db, kt_ops.linear_backward_workspace(M, K, N))  # x as the gradient
    _, _, dwx, tw, dbx, tb = ref.linear_backward(x, y, dw, dt)
    near(dw, dwx, tw)
    near(db, dbx, tb)


@pytest.mark.parametrize("M,D,F", [(1, 4304, 64), (5, 2304, 1152), (33, 5120, 40), (128, 8192, 264), (200, 4096, 320)])
@pytest.mark.parametrize("dtype,bias", [("f16", True), ("bf16", False)])
def test_gated_projection_of_few_tiles_with_long_sums(M, D, F, dtype, bias):
    g = torch.Generator().manual_seed(2 * M + D + F)
    dt, name = DT[dtype], sorted(ACTS)[(M + F) % len(ACTS)]
    x, w = randn(g, M, D, dtype=dt, pad=24), randn(g, 2 * F, D, dtype=dt, std=D ** -0.5)
    b = randn(g, 2 * F, dtype=dt, std=0.2) if bias else None
    hs, h = nans(M, F, dt, 8)
    ps, p = nans(M, 2 * F, dt, 16)
    kt_ops.kt_glu_forward(x, w, b, h, p, ACTS[name])
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    hx, th, px, tp = ref.glu(x, w, b, name, dt)
    near(p, px, tp)
    near(h, hx, th)
    assert hs[:, F:].isnan().all() and ps[:, 2 * F:].isnan().all()
    alone = torch.empty_like(h)
    kt_ops.kt_glu_forward(x, w, b, alone, None, ACTS[name])
    assert torch.equal(alone, h)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 31, 100, 127, 128, 129])
@pytest.mark.parametrize("N", [8, 24, 64, 120, 136])
def test_rows_and_columns_that_end_inside_a_tile(M, N):
    """What a tile reads beyond its operands may be anything, NaN too: none of it reaches a result."""
    dt, K = torch.bfloat16, 328
    g = torch.Generator().manual_seed(M + N)
    junk = torch.full((4096, 4096), float("nan"), dtype=dt, device="cuda")
    kt_ops.kt_linear_forward(junk, junk, None, torch.empty_like(junk))  # NaN in every block's shared memory
    x, w, b = randn(g, M, K, dtype=dt), randn(g, N, K, dtype=dt, std=K ** -0.5), randn(g, N, dtype=dt)
    ys, y = nans(M, N, dt, 8)
    kt_ops.kt_linear_forward(x, w, b, y)
    yx, ty = ref.product(x.double(), w.double(), b)
    near(y, yx, ref.rounded(yx, ty, dt))
    assert ys[:, N:].isnan().all()


@pytest.mark.parametrize("M", [3, 128])
def test_a_wait_that_runs_out_in_a_shared_gated_tile_shows(M):
    """Few tiles with long sums: one CTA of a cluster gives up, and its tile shows it."""
    g = torch.Generator().manual_seed(M)
    D, F, dt = 4096, 200, torch.bfloat16
    x, w, b = randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=0.02), randn(g, 2 * F, dtype=dt)
    want, got = torch.empty(M, F, dtype=dt, device="cuda"), torch.full((M, F), 7.0, dtype=dt, device="cuda")
    p, q = torch.empty(M, 2 * F, dtype=dt, device="cuda"), torch.full((M, 2 * F), 7.0, dtype=dt, device="cuda")
    kt_ops.kt_glu_forward(x, w, b, want, p, kt_mlp.KT_ACT_SILU)
    kt_ops.kt_matmul_debug_stall(True, 20000)
    try:
        kt_ops.kt_glu_forward(x, w, b, got, q, kt_mlp.KT_ACT_SILU)
        assert kt_ops.kt_matmul_status() == kt_mlp.KT_ERR_TIMEOUT
    finally:
        kt_ops.kt_matmul_debug_stall(False)
    for a, c in ((got, want), (q, p)):
        assert a[0, 0].isnan() and (a.isnan() | (a == c)).all()
    kt_ops.kt_glu_forward(x, w, b, got, q, kt_mlp.KT_ACT_SILU)
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK and torch.equal(got, want) and torch.equal(q, p)


def test_a_workspace_of_two_graphs_replayed_in_turn():
    """Both graphs' gradients are those of the inputs at each replay, whichever ran before."""
    g = torch.Generator().manual_seed(9)
    dt = torch.float16
    sizes = [(300, 264, 520), (4096, 72, 136)]
    ws = max((kt_ops.glu_backward_workspace(*s) for s in sizes), key=lambda t: t.numel())
    calls = []
    for M, D, F in sizes:
        x, w = randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=D ** -0.5)
        p, dh = randn(g, M, 2 * F, dtype=dt), randn(g, M, F, dtype=dt, std=0.5)
        out = torch.empty(M, D, dtype=dt, device="cuda"), torch.empty(2 * F, D, dtype=dt, device="cuda"), torch.empty(2 * F, device="cuda")
        run = lambda x=x, w=w, p=p, dh=dh, out=out: kt_ops.kt_glu_backward(dh, p, x, w, *out, kt_mlp.KT_ACT_GELU_TANH, ws)
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        calls.append((graph, out, [t.clone() for t in out]))
    for i in (0, 1, 1, 0, 1, 0):
        graph, out, want = calls[i]
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        for t, u in zip(out, want):
            assert torch.equal(t, u)
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK


@pytest.mark.parametrize("M,N,K", [(700, 5000, 1288), (16384, 1280, 2560), (331, 640, 2560), (64, 2560, 264)])
def test_a_wait_that_runs_out_in_a_linear_layers_gradients_shows(M, N, K):
    """The first block stalls for 20 ms and raises no flag for its partial sums: the blocks that add them give up their
    tiles.  What could not be computed is NaN, all else is as it is without the stall, and the next call is right."""
    g = torch.Generator().manual_seed(M + N)
    dt = torch.bfloat16
    x, w, dy = randn(g, M, K, dtype=dt), randn(g, N, K, dtype=dt, std=K ** -0.5), randn(g, M, N, dtype=dt, std=0.25)
    ws = kt_ops.linear_backward_workspace(M, N, K)

    def run(bias):
        out = torch.full((M, K), 7.0, dtype=dt, device="cuda"), torch.full((N, K), 7.0, dtype=dt, device="cuda")
        kt_ops.kt_linear_backward(dy, x, w, *out, torch.empty(N, device="cuda") if bias else None, ws)
        return out

    for bias in (False, True):
        want = run(bias)
        assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
        kt_ops.kt_matmul_debug_stall(True, 20000)
        try:
            got = run(bias)
            assert kt_ops.kt_matmul_status() == kt_mlp.KT_ERR_TIMEOUT
        finally:
            kt_ops.kt_matmul_debug_stall(False)
        assert any(a.isnan().any() for a in got)
        for a, b in zip(got, want):
            assert (a.isnan() | (a == b)).all()
        for a, b in zip(run(bias), want):
            assert torch.equal(a, b)
        assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK


@pytest.mark.parametrize("M,D,F", [(729, 1152, 4304), (5000, 264, 2560), (4096, 640, 2560)])
def test_a_wait_that_runs_out_in_a_gated_blocks_gradients_shows(M, D, F):
    g = torch.Generator().manual_seed(M)
    dt = torch.float16
    x, w = randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=D ** -0.5)
    p, dh = randn(g, M, 2 * F, dtype=dt), randn(g, M, F, dtype=dt, std=0.5)
    ws = kt_ops.glu_backward_workspace(M, D, F)

    def run():
        out = torch.full((M, D), 7.0, dtype=dt, device="cuda"), torch.full((2 * F, D), 7.0, dtype=dt, device="cuda"), torch.empty(2 * F, device="cuda")
        kt_ops.kt_glu_backward(dh, p, x, w, *out, kt_mlp.KT_ACT_SILU, ws)
        return out

    want = run()
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    kt_ops.kt_matmul_debug_stall(True, 20000)
    try:
        got = run()
        assert kt_ops.kt_matmul_status() == kt_mlp.KT_ERR_TIMEOUT
    finally:
        kt_ops.kt_matmul_debug_stall(False)
    assert got[0].isnan().any() or got[1].isnan().any()
    for a, b in zip(got, want):
        assert (a.isnan() | (a == b)).all()
    assert torch.equal(got[2], want[2])  # the bias gradient hangs on neither product
    for a, b in zip(run(), want):
        assert torch.equal(a, b)
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK


# sizes whose last tiles' steps are shared out, joined behind flags in the workspace (checked by the flags that were raised)
def gated_gradients(M, D, F, dt, g, bias, ws):
    """(inputs, outputs, call) of a gated block's gradients."""
    x, w = randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=D ** -0.5)
    p, dh = randn(g, M, 2 * F, dtype=dt), randn(g, M, F, dtype=dt, std=0.5)
    out = [torch.empty(M, D, dtype=dt, device="cuda"), torch.empty(2 * F, D, dtype=dt, device="cuda")]
    db = torch.empty(2 * F, device="cuda") if bias else None
    return [dh, p, x, w], out + [db] * bias, lambda ws=ws: kt_ops.kt_glu_backward(dh, p, x, w, *out, db, kt_mlp.KT_ACT_GELU_TANH, ws)


def linear_gradients(M, N, K, dt, g, bias, ws):
    x, w, dy = randn(g, M, K, dtype=dt), randn(g, N, K, dtype=dt, std=K ** -0.5), randn(g, M, N, dtype=dt, std=0.25)
    out = [torch.empty(M, K, dtype=dt, device="cuda"), torch.empty(N, K, dtype=dt, device="cuda")]
    db = torch.empty(N, device="cuda") if bias else None
    return [dy, x, w], out + [db] * bias, lambda ws=ws: kt_ops.kt_linear_backward(dy, x, w, *out, db, ws)


SHARED = [(gated_gradients, (729, 1152, 4304)), (gated_gradients, (5000, 264, 2560)), (linear_gradients, (700, 5000, 1288)),
          (linear_gradients, (16384, 1280, 2560))]


def room(make, size):
    return (kt_ops.glu_backward_workspace if make is gated_gradients else kt_ops.linear_backward_workspace)(*size)


def renew(inputs, g):
    for t in inputs:
        t.copy_(torch.randn(t.shape, generator=g, dtype=torch.float32, device="cuda") * 0.2)


@pytest.mark.parametrize("bias", [False, True])
def test_shared_gradients_of_graphs_with_one_workspace(bias):
    """New values before each replay, another graph in between, whose flags and partial sums stay in the workspace: each
    replay's results are those of a call of its own with a workspace of its own, bit for bit."""
    g, gd = torch.Generator().manual_seed(3), torch.Generator(device="cuda").manual_seed(3)
    ws = max((room(*s) for s in SHARED), key=lambda t: t.numel())
    ws.fill_(255)
    calls = []
    for make, size in SHARED:
        inputs, out, run = make(*size, torch.bfloat16, g, bias, ws)
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        calls.append((graph, inputs, out, run, room(make, size)))
    for i in (0, 1, 1, 2, 0, 3, 2, 2, 3, 1, 0):
        graph, inputs, out, run, own = calls[i]
        renew(inputs, gd)
        run(own.fill_(0))
        want = [t.clone() for t in out]
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        for t, u in zip(out, want):
            assert torch.equal(t, u), i
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK


@pytest.mark.parametrize("make,size", SHARED)
def test_shared_gradients_again_and_again_into_the_same_buffers(make, size):
    """Values written anew right before each of ten steps, eager and in one graph."""
    g, gd = torch.Generator().manual_seed(4), torch.Generator(device="cuda").manual_seed(4)
    ws = room(make, size)
    inputs, out, run = make(*size, torch.float16, g, True, ws)
    new = []
    for _ in range(3):
        renew(inputs, gd)
        new.append([t.clone() for t in inputs])
    want = []
    for n in new:
        for t, u in zip(inputs, n):
            t.copy_(u)
        torch.cuda.synchronize()
        run(room(make, size))
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    got = [[torch.empty_like(t) for t in out] for _ in range(10)]

    def steps():
        for i, to in enumerate(got):
            for t, u in zip(inputs, new[i % 3]):
                t.copy_(u)
            run()
            for t, u in zip(to, out):
                t.copy_(u)

    def check():
        torch.cuda.synchronize()
        assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
        for i, to in enumerate(got):
            for t, u in zip(to, want[i % 3]):
                assert torch.equal(t, u), i
                t.fill_(float("nan"))

    steps()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(2):
        graph.replay()
        check()


def test_shared_gradients_on_three_streams_at_once():
    g = torch.Generator().manual_seed(5)
    calls = []
    for make, size in SHARED[:3]:
        ws = room(make, size)
        inputs, out, run = make(*size, torch.bfloat16, g, True, ws)
        run()
        torch.cuda.synchronize()
        calls.append((out, [t.clone() for t in out], run, torch.cuda.Stream()))
    for _ in range(20):
        for out, _, run, stream in calls:
            with torch.cuda.stream(stream):
                run()
    torch.cuda.synchronize()
    assert kt_ops.kt_matmul_status() == kt_mlp.KT_OK
    for out, want, _, _ in calls:
        for t, u in zip(out, want):
            assert torch.equal(t, u)


@pytest.mark.parametrize("M", [40, 729])
def test_gradients_below_the_normal_numbers(M):
    """Gradients near 1e-6 in float16: dp is held to 2^-25 in absolute terms, and all of it that is below is lost.  The same
    gradients under a loss scale of 2^10 keep what dh has."""
    g = torch.Generator().manual_seed(M)
    D, F, dt = 264, 520, torch.float16
    x, w = randn(g, M, D, dtype=dt), randn(g, 2 * F, D, dtype=dt, std=D ** -0.5)
    p, dh = randn(g, M, 2 * F, dtype=dt), randn(g, M, F, dtype=dt, std=1e-6)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(2 * F, device="cuda")
    off = []
    for scale in (1.0, 1024.0):
        scaled = dh * scale  # exact: dh is a multiple of 2^-24
        kt_ops.kt_glu_backward(scaled, p, x, w, dx, dw, db, kt_mlp.KT_ACT_SILU, kt_ops.glu_backward_workspace(M, D, F))
        dxx, tx, dwx, tw, dbx, tb = ref.glu_backward(scaled, p, x, w, "silu", dt)
        near(dx, dxx, tx)
        near(dw, dwx, tw)
        near(db, dbx, tb)
        off.append(((dw.double() - dwx).norm() / dwx.norm()).item())
    assert off[1] < off[0] / 4
    # columns whose elements of dp are all below 2^-25 are lost, but not to the bias gradient
    p[:, F:] = -40.0
    dh.fill_(2.0 ** -10)
    kt_ops.kt_glu_backward(dh, p, x, w, dx, dw, db, kt_mlp.KT_ACT_SILU, kt_ops.glu_backward_workspace(M, D, F))
    assert not dx.any() and not dw.any() and db.all()
