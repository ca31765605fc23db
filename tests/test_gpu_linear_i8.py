"""8-bit rows and the 8-bit linear layer on the GPU: the integers exactly, the products within
the few roundings that the definition has."""
import pytest
import torch

from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops

import ops_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTS = {"geglu": kt_mlp.KT_ACT_GEGLU, "gelu_erf": kt_mlp.KT_ACT_GELU_ERF, "gelu_tanh": kt_mlp.KT_ACT_GELU_TANH,
        "gelu_sigmoid": kt_mlp.KT_ACT_GELU_SIGMOID, "silu": kt_mlp.KT_ACT_SILU}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_mlp_gemms_gb300 import build
    build.build()
    kt_ops.load()


def quantize(x, K, act=kt_mlp.KT_ACT_NONE, pad=0):
    M = x.shape[0]
    q = torch.full((M, K + pad), 99, dtype=torch.int8, device="cuda")[:, :K]
    scale = torch.full((M,), -1.0, device="cuda")
    kt_ops.kt_quantize_rows(x, q, scale, act)
    return q, scale


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,pad", [(1, 1, 0), (3, 16, 0), (5, 37, 3), (9, 640, 0), (729, 1152, 0), (33, 1280, 8), (8, 2048, 16),
                                     (7, 4304, 0), (5, 10240, 0), (3, 16384, 0), (2, 16381, 0), (4000, 72, 0)])
def test_the_integers_are_the_nearest(M, K, pad, dtype):
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn(M, K + pad, generator=g) * torch.exp(3 * torch.randn(M, 1, generator=g))).to(DT[dtype]).cuda()[:, :K]
    q, scale = quantize(x, K, pad=pad)
    qx, sx = ref.quantize(x)
    assert torch.equal(q, qx)
    assert torch.equal(scale.nan_to_num(-7.0), sx.nan_to_num(-7.0))  # a float16 row may overflow: no number on both sides


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_ties_zeros_subnormals_and_bad_rows(dtype):
    dt = DT[dtype]
    K = 256
    ties = torch.arange(K, dtype=torch.float32) - 127.5  # scale 1 with 127 put first: every value but it a tie
    x = torch.zeros(8, K)
    x[0], x[0, 0] = ties.clamp(-126.5, 126.5), 127.0
    x[2, 5] = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps  # the smallest subnormal, alone
    x[3] = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps * (torch.arange(K) - 100)
    x[4], x[4, 9] = ties, float("nan")
    x[5], x[5, 255] = ties, float("-inf")
    x[6] = torch.finfo(dt).max
    x[7] = 1e-5 * ties
    x = x.to(dt).cuda()
    q, scale = quantize(x, K)
    qx, sx = ref.quantize(x)
    assert torch.equal(q, qx)
    assert torch.equal(scale.nan_to_num(-7.0), sx.nan_to_num(-7.0))
    assert scale[1] == 0 and scale[4].isnan() and scale[5].isnan() and (q[6] == 127).all()


@pytest.mark.parametrize("name", sorted(ACTS))
@pytest.mark.parametrize("M,K", [(5, 72), (33, 1280), (3, 5120), (9, 101)])
def test_activations_as_they_are_quantised(name, M, K):
    """The activation is good to 2e-5 (the library's tested bound), so a value may be off by that
    and by half a step of its row's scale, which itself carries 2e-5."""
    g = torch.Generator().manual_seed(K)
    x = (2 * torch.randn(M, 2 * K if name == "geglu" else K, generator=g)).to(torch.bfloat16).cuda()
    q, scale = quantize(x, K, ACTS[name])
    v = ref.act(x.double(), name)
    most = v.abs().amax(1)
    assert ((scale.double() * 127 - most).abs() <= 2.1e-5 * most).all()
    assert ((q.double() * scale.double()[:, None] - v).abs() <= scale.double()[:, None] * 0.5001 + 2.1e-5 * v.abs() + 1e-37).all()


SHAPES = [(1, 1, 16), (1, 8, 64), (3, 33, 48), (4, 10240, 1280), (7, 100, 4112), (8, 640, 640), (9, 31, 64), (16, 257, 144),
          (33, 64, 1152), (64, 512, 8192), (100, 130, 272), (127, 1000, 640), (128, 256, 128), (129, 255, 2048), (300, 4304, 1152),
          (729, 1152, 4304), (1000, 520, 80), (2048, 72, 96),
          # several tiles per pair of each width
          (1100, 4304, 272), (3000, 12800, 80), (1300, 10240, 144), (2000, 5000, 208), (140, 9728, 640), (5000, 640, 144)]


@pytest.mark.parametrize("dtype,bias", [("f16", False), ("bf16", True)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(M, N, K, dtype, bias):
    g = torch.Generator().manual_seed(M * 7 + N * 3 + K)
    dt = DT[dtype]
    q = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    sx, sw = (torch.rand(M, generator=g) * 1e-3).cuda(), (torch.rand(N, generator=g) * 1e-2).cuda()
    b = torch.randn(N, generator=g).to(dt).cuda() if bias else None
    y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    kt_ops.kt_linear_i8(q, sx, w, sw, b, y)
    yx, tol = ref.linear_i8(q, sx, w, sw, b)
    bad = ~((y.double() - yx).abs() <= tol + ref.half(dt) * yx.abs() + ref.floor(dt))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), y[bad][0].item(), yx[bad][0].item())


@pytest.mark.parametrize("M", [5, 70, 300])
def test_products_of_slices(M):
    """Pitches wider than the rows, an odd pitch of Y, and what lies outside stays untouched."""
    g = torch.Generator().manual_seed(M)
    N, K = 203, 208
    q = torch.randint(-127, 128, (M, K + 32), generator=g, dtype=torch.int32).to(torch.int8).cuda()[:, :K]
    w = torch.randint(-127, 128, (N, K + 48), generator=g, dtype=torch.int32).to(torch.int8).cuda()[:, :K]
    sx, sw = torch.rand(M, generator=g).cuda() * 1e-3, torch.rand(N, generator=g).cuda() * 1e-2
    whole = torch.full((M, N + 6), 7.0, dtype=torch.bfloat16, device="cuda")
    kt_ops.kt_linear_i8(q, sx, w, sw, None, whole[:, 3:3 + N])
    yx, tol = ref.linear_i8(q, sx, w, sw, None)
    assert ((whole[:, 3:3 + N].double() - yx).abs() <= tol + ref.half(torch.bfloat16) * yx.abs()).all()
    assert (whole[:, :3] == 7).all() and (whole[:, 3 + N:] == 7).all()


@pytest.mark.parametrize("M", [8, 200])
@pytest.mark.parametrize("K", [1024, 4096])
def test_the_largest_sums(M, K):
    """All values -128 or 127 with equal signs: sums up to 2^26.  Exact for K up to 1024 at any
    M and for any K at few tokens; above, an fp32 sum of K / 16 steps, each off by 2^-23 at most."""
    N = 96
    q = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    q[1::3] = 127
    one, step = torch.ones(M, device="cuda"), torch.full((N,), 2.0 ** -20, device="cuda")
    y = torch.empty(M, N, dtype=torch.float16, device="cuda")
    kt_ops.kt_linear_i8(q, one, w, step, None, y)
    yx, tol = ref.linear_i8(q, one, w, step, None)
    extra = 0.0 if M <= 8 or K <= 1024 else K / 16 * 2.0 ** -23
    assert ((y.double() - yx).abs() <= tol + (ref.half(torch.float16) + extra) * yx.abs()).all()


@pytest.mark.parametrize("M", [8, 100, 300])
def test_sums_that_cancel_are_exact(M):
    """Partial sums of 2^23 that come back to small integers, which float16 holds: not one unit lost."""
    g = torch.Generator().manual_seed(M)
    N, half = 80, 512
    sign = torch.randint(0, 2, (1, half), generator=g) * 2 - 1
    q1 = (127 * sign).expand(M, half).clone()
    w1 = (127 * sign).expand(N, half).clone()
    back = -w1
    for n in range(N):  # up to 15 entries of the second half are off by one
        at = torch.randperm(half, generator=g)[:n % 16]
        back[n, at] += -back[n, at].sign()
    q = torch.cat([q1, q1], 1).to(torch.int8).cuda()
    w = torch.cat([w1, back], 1).to(torch.int8).cuda()
    q[:, 3] = torch.randint(-127, 128, (M,), generator=g, dtype=torch.int32).to(torch.int8).cuda()  # rows differ
    q[:, half + 3] = q[:, 3]
    y = torch.empty(M, N, dtype=torch.float16, device="cuda")
    kt_ops.kt_linear_i8(q, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), None, y)
    exact = q.cpu().long() @ w.cpu().long().t()
    assert exact.abs().max() <= 2048 and exact.unique().numel() > 10
    assert torch.equal(y.cpu().long(), exact)


def test_quantised_layer_in_a_graph_and_on_another_stream():
    g = torch.Generator().manual_seed(3)
    M, N, K = 200, 320, 640
    x = torch.randn(M, K, generator=g).half().cuda()
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    sw = torch.rand(N, generator=g).cuda() * 1e-2
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")

    def step(y):
        kt_ops.kt_quantize_rows(x, q, s)
        kt_ops.kt_linear_i8(q, s, w, sw, None, y)

    eager, captured, side = (torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda") for _ in range(3))
    step(eager)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(eager, captured) and torch.equal(eager, side)


def test_no_tokens():
    e = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    q, s = torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    kt_ops.kt_quantize_rows(e, q, s)
    kt_ops.kt_linear_i8(q, s, torch.zeros(8, 64, dtype=torch.int8, device="cuda"), torch.zeros(8, device="cuda"), None,
                        torch.empty(0, 8, dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,bias", [("f16", True), ("bf16", False)])
@pytest.mark.parametrize("M,N,K", [(17, 1280, 5120), (100, 8192, 8192), (127, 131, 1168), (129, 520, 4304), (256, 512, 8192), (257, 510, 4112),
                                   (729, 1152, 4304), (20, 8, 16384), (500, 65, 2064), (128, 640, 1040)])
def test_long_rows_of_few_tiles(M, N, K, dtype, bias):
    """Tiles whose steps are shared out: against the definition, at an odd pitch, and the same bits again."""
    g = torch.Generator().manual_seed(M + N + K)
    dt = DT[dtype]
    q = torch.randint(-127, 128, (M, K + 16), generator=g, dtype=torch.int32).to(torch.int8).cuda()[:, :K]
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    sx, sw = (torch.rand(M, generator=g) * 1e-3).cuda(), (torch.rand(N, generator=g) * 1e-2).cuda()
    b = torch.randn(N, generator=g).to(dt).cuda() if bias else None
    yx, tol = ref.linear_i8(q, sx, w, sw, b)
    for pad in (0, 3):
        whole = torch.full((M, N + pad), 7.0, dtype=dt, device="cuda")
        kt_ops.kt_linear_i8(q, sx, w, sw, b, whole[:, :N])
        y = whole[:, :N]
        bad = ~((y.double() - yx).abs() <= tol + ref.half(dt) * yx.abs() + ref.floor(dt))
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), y[bad][0].item(), yx[bad][0].item())
        assert (whole[:, N:] == 7).all()
        again = torch.empty_like(whole)[:, :N]
        kt_ops.kt_linear_i8(q, sx, w, sw, b, again)
        assert torch.equal(again, y)


def test_long_rows_captured_and_on_another_stream():
    g = torch.Generator().manual_seed(5)
    M, N, K = 40, 640, 4096
    q = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    sx, sw = (torch.rand(M, generator=g) * 1e-3).cuda(), (torch.rand(N, generator=g) * 1e-2).cuda()
    y = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    z = torch.full_like(y, float("nan"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            kt_ops.kt_linear_i8(q, sx, w, sw, None, y)
    graph.replay()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kt_ops.kt_linear_i8(q, sx, w, sw, None, z)
    torch.cuda.synchronize()
    yx, tol = ref.linear_i8(q, sx, w, sw, None)
    assert ((y.double() - yx).abs() <= tol + ref.half(torch.float16) * yx.abs() + ref.floor(torch.float16)).all()
    assert torch.equal(y, z)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("M,N,K", [(4, 1280, 640), (16, 520, 1296), (64, 640, 4096), (300, 520, 272), (729, 4304, 640)])
def test_new_values_in_the_same_buffers_are_read(M, N, K, captured):
    """Tokens and weights quantised into the same buffers again and again, each product right behind
    its operands' writes: every step's result is that of the step alone, bit for bit."""
    g = torch.Generator().manual_seed(M + K)
    steps = 12
    x = (torch.randn(steps, M, K, generator=g) * torch.exp(torch.randn(steps, M, 1, generator=g))).to(torch.bfloat16).cuda()
    wf = (torch.randn(steps, N, K, generator=g) / K ** 0.5).to(torch.bfloat16).cuda()

    def buffers():
        return (torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda"),
                torch.zeros(N, K, dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda"))

    def step(i, b, y):
        kt_ops.kt_quantize_rows(wf[i], b[2], b[3])
        kt_ops.kt_quantize_rows(x[i], b[0], b[1])
        kt_ops.kt_linear_i8(*b, None, y)

    alone = torch.full((steps, M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i in range(steps):
        b = buffers()
        step(i, b, alone[i])
        torch.cuda.synchronize()
        qx, sx = ref.quantize(x[i])
        assert torch.equal(b[0], qx) and torch.equal(b[1], sx)
        yx, tol = ref.linear_i8(*b, None)
        assert ((alone[i].double() - yx).abs() <= tol + ref.half(torch.bfloat16) * yx.abs()).all()
    b = buffers()
    got = torch.full_like(alone, float("nan"))
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(steps):
                step(i, b, got[i])
        graph.replay()
        torch.cuda.synchronize()
        got.fill_(float("nan"))
        graph.replay()
    else:
        for i in range(steps):
            step(i, b, got[i])
    torch.cuda.synchronize()
    for i in range(steps):
        assert torch.equal(got[i], alone[i]), i


# one CTA per tile of both widths, a pair per tile of each width, clusters that share a tile
@pytest.mark.parametrize("M,N,K", [(100, 130, 272), (100, 1500, 272), (140, 9728, 640), (5000, 640, 144), (1300, 10240, 144), (2000, 5000, 208),
                                   (64, 1280, 5120), (100, 8192, 4096)])
def test_a_wait_that_runs_out_is_reported_and_shows(M, N, K):
    """The first block waits, for 20 ms, on a barrier that nobody signals: the status says so, its tiles
    are NaN and nothing is left unwritten, and the next call is right again."""
    g = torch.Generator().manual_seed(M)
    q = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    sx, sw = (torch.rand(M, generator=g) * 1e-3).cuda(), (torch.rand(N, generator=g) * 1e-2).cuda()
    want = torch.empty(M, N, dtype=torch.float16, device="cuda")
    kt_ops.kt_linear_i8(q, sx, w, sw, None, want)
    assert kt_ops.kt_linear_i8_status() == kt_mlp.KT_OK
    got = torch.full((M, N + 3), 7.0, dtype=torch.float16, device="cuda")
    kt_ops.kt_linear_i8_debug_stall(True, 20000)
    try:
        kt_ops.kt_linear_i8(q, sx, w, sw, None, got[:, :N])
        assert kt_ops.kt_linear_i8_status() == kt_mlp.KT_ERR_TIMEOUT
    finally:
        kt_ops.kt_linear_i8_debug_stall(False)
    bad = got[:, :N].isnan()
    assert bad[0, 0] and (bad | (got[:, :N] == want)).all()
    assert (got[:, N:] == 7).all()
    assert kt_ops.kt_linear_i8_status() == kt_mlp.KT_OK
    kt_ops.kt_linear_i8(q, sx, w, sw, None, got[:, :N])
    assert kt_ops.kt_linear_i8_status() == kt_mlp.KT_OK
    assert torch.equal(got[:, :N], want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("K", [64, 1024])
def test_a_row_is_the_same_in_calls_of_any_length(K, dtype):
    """Exact sums, then the same roundings: on the integer products of few tokens, on one tile and on
    many."""
    g = torch.Generator().manual_seed(K)
    N, dt = 10240, DT[dtype]
    q = torch.randint(-128, 128, (300, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    sx, sw = (torch.rand(300, generator=g) * 1e-3).cuda(), (torch.rand(N, generator=g) * 1e-2).cuda()
    b = torch.randn(N, generator=g).to(dt).cuda()
    first = torch.empty(16, N, dtype=dt, device="cuda")
    kt_ops.kt_linear_i8(q[:16], sx[:16], w, sw, b, first)
    for M in (1, 17, 130, 300):
        y = torch.empty(M, N, dtype=dt, device="cuda")
        kt_ops.kt_linear_i8(q[:M], sx[:M], w, sw, b, y)
        assert torch.equal(y[:16], first[:M])
