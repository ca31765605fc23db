"""The mixture-of-experts layer for a few tokens on the GPU against the 64-bit definition: the
same experts, and outputs within a bound that follows the kernel's steps (ops_reference.moe)."""
import pytest
import torch

from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops

import ops_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f16": (torch.float16, kt_mlp.KT_F16), "bf16": (torch.bfloat16, kt_mlp.KT_BF16)}
ACTS = {"geglu": kt_mlp.KT_ACT_GEGLU, "gelu_erf": kt_mlp.KT_ACT_GELU_ERF, "gelu_tanh": kt_mlp.KT_ACT_GELU_TANH,
        "gelu_sigmoid": kt_mlp.KT_ACT_GELU_SIGMOID, "silu": kt_mlp.KT_ACT_SILU, "none": kt_mlp.KT_ACT_NONE}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_mlp_gemms_gb300 import build
    build.build()
    kt_ops.load()


def problem(T, D, F, E, k, act, dtype, bias, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype][0]
    up = 2 * F if act == "geglu" else F

    def r(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dt).cuda()

    t = {"X": r(T, D + pad)[:, :D], "W_router": r(E, D, std=D ** -0.5), "W_up": r(E, up, D, std=D ** -0.5),
         "W_down": r(E, D, F, std=F ** -0.5), "b_up": r(E, up, std=0.14) if bias else None,
         "b_down": r(E, D, std=0.14) if bias else None}
    return t


def plan_of(T, D, F, E, k, act, dtype, bias, normalize):
    return kt_ops.MoePlan(T, D, F, E, k, ACTS[act], DT[dtype][1], bias=bias, normalize=normalize)


def run(plan, t, R=None, Y=None):
    T, D = t["X"].shape
    Y = torch.full((T, D), float("nan"), dtype=t["X"].dtype, device="cuda") if Y is None else Y
    ids = torch.full((T, plan.top_k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, plan.top_k), float("nan"), device="cuda")
    plan.run(t["X"], t["W_router"], t["W_up"], t["W_down"], Y, t["b_up"], t["b_down"], R=R, ids=ids, weights=w)
    assert plan.status() == kt_mlp.KT_OK
    return Y, ids, w


def reference(t, R, k, act, normalize):
    def f(x, name):
        return x if name == "none" else ref_act(x, name)
    ref_act, ref.act = ref.act, f
    try:
        return ref.moe(t["X"], t["W_router"], t["W_up"], t["W_down"], t["b_up"], t["b_down"], R, k, act, normalize, t["X"].dtype)
    finally:
        ref.act = ref_act


def check(got, want):
    Y, ids, w = got
    y, ex, wx, tol = want
    assert torch.equal(ids.long(), ex)
    assert ((w.double() - wx).abs() <= 64 * ref.U * wx).all()
    bad = ~((Y.double() - y).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), Y[bad][0].item(), y[bad][0].item(), tol[bad][0].item())


CASES = [
    # T, D, F, E, k, act, dtype, bias, normalize, residual, pad
    (1, 8, 8, 1, 1, "none", "f16", False, True, False, 0),
    (1, 64, 64, 8, 2, "geglu", "bf16", False, True, False, 0),
    (1, 1280, 640, 8, 2, "geglu", "bf16", True, False, True, 0),
    (2, 72, 136, 4, 4, "silu", "f16", True, True, False, 8),
    (7, 264, 520, 5, 3, "gelu_erf", "f16", True, False, True, 0),
    (8, 256, 1000, 16, 2, "gelu_tanh", "bf16", False, True, False, 0),
    (9, 320, 648, 16, 2, "geglu", "f16", True, True, True, 16),
    (16, 200, 72, 2, 2, "gelu_sigmoid", "f16", True, True, False, 0),
    (17, 128, 264, 3, 1, "geglu", "bf16", True, False, False, 0),
    (33, 96, 104, 256, 16, "silu", "bf16", False, True, False, 0),
    (64, 64, 136, 2, 2, "geglu", "f16", True, True, True, 0),
    (64, 136, 72, 64, 8, "gelu_erf", "bf16", True, False, False, 0),
    (64, 1152, 304, 40, 6, "geglu", "bf16", False, True, False, 0),
    (5, 2560, 64, 33, 1, "gelu_tanh", "f16", False, False, False, 0),
    (3, 64, 8192, 6, 2, "geglu", "bf16", True, True, False, 0),
]


@pytest.mark.parametrize("T,D,F,E,k,act,dtype,bias,normalize,residual,pad", CASES)
def test_layer(T, D, F, E, k, act, dtype, bias, normalize, residual, pad):
    t = problem(T, D, F, E, k, act, dtype, bias, 100 * T + D + F, pad)
    R = problem(T, D, F, E, k, act, dtype, False, 5)["X"] if residual else None
    plan = plan_of(T, D, F, E, k, act, dtype, bias, normalize)
    first = run(plan, t, R)
    check(first, reference(t, R, k, act, normalize))
    again = run(plan, t, R)  # the counters are back at zero, the sums in the same order
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_fewer_tokens_than_the_plan_is_for():
    plan = plan_of(64, 128, 192, 8, 2, "geglu", "bf16", False, True)
    t = problem(64, 128, 192, 8, 2, "geglu", "bf16", False, 1)
    for T in (64, 1, 20, 9, 3):
        u = {**t, "X": t["X"][:T]}
        check(run(plan, u), reference(u, None, 2, "geglu", True))
    empty = {**t, "X": t["X"][:0]}
    plan.run(empty["X"], t["W_router"], t["W_up"], t["W_down"], torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("T", [5, 64])
def test_equal_logits_go_to_the_lower_experts(T):
    t = problem(T, 256, 64, 12, 3, "silu", "f16", False, 2)
    t["W_router"][:] = t["W_router"][:1].clone()  # every expert has the same logit
    plan = plan_of(T, 256, 64, 12, 3, "silu", "f16", False, True)
    Y, ids, w = run(plan, t)
    assert (ids == torch.arange(3, device="cuda", dtype=torch.int32)).all()
    check((Y, ids, w), reference(t, None, 3, "silu", True))


def test_every_token_with_the_same_expert():
    t = problem(64, 128, 136, 16, 1, "geglu", "bf16", True, 3)
    t["X"][:] = t["X"][:1].clone()
    plan = plan_of(64, 128, 136, 16, 1, "geglu", "bf16", True, False)
    Y, ids, w = run(plan, t)
    check((Y, ids, w), reference(t, None, 1, "geglu", False))
    assert (Y == Y[:1]).all()


def test_logits_that_differ_far_below_fp32():
    """Two experts whose logits agree to about 2^-36: the order is that of the exact sums."""
    D = 64
    t = problem(4, D, 64, 2, 1, "silu", "bf16", False, 4)
    t["W_router"][:] = 0
    t["X"][:] = 0
    t["X"][:, 0], t["X"][:, 1] = 256.0, 2.0 ** -14
    t["W_router"][:, 0] = 256.0
    t["W_router"][1, 1] = 2.0 ** -6  # expert 1 is ahead by 2^-20 on 2^16
    plan = plan_of(4, D, 64, 2, 1, "silu", "bf16", False, True)
    _, ids, _ = run(plan, t)
    assert (ids == 1).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_token_spoils_itself_alone(value):
    t = problem(12, 128, 64, 8, 2, "geglu", "bf16", False, 6)
    plan = plan_of(12, 128, 64, 8, 2, "geglu", "bf16", False, True)
    clean, _, _ = run(plan, t)
    t["X"] = t["X"].clone()
    t["X"][7, 3] = value
    Y, ids, w = run(plan, t)
    assert not Y[7].isfinite().any()
    assert (0 <= ids[7]).all() and (ids[7] < 8).all() and ids[7, 0] != ids[7, 1]
    keep = [r for r in range(12) if r != 7]
    assert torch.equal(Y[keep], clean[keep])


def test_in_place_graph_and_another_stream():
    t = problem(9, 256, 264, 8, 2, "geglu", "bf16", True, 7)
    plan = plan_of(9, 256, 264, 8, 2, "geglu", "bf16", True, True)
    X = t["X"].clone()
    want, _, _ = run(plan, t, R=X)
    t["X"] = X.clone()
    got, _, _ = run(plan, t, R=t["X"], Y=t["X"])  # the residual stream, updated in place
    assert torch.equal(got, want)
    t["X"] = X.clone()
    side, captured = torch.empty_like(X), torch.empty_like(X)
    args = (t["W_router"], t["W_up"], t["W_down"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        plan.run(t["X"], *args, side, t["b_up"], t["b_down"], R=X)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(t["X"], *args, captured, t["b_up"], t["b_down"], R=X)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(side, want) and torch.equal(captured, want)


def test_refusals_of_a_run():
    t = problem(4, 64, 64, 8, 2, "silu", "f16", False, 8)
    plan = plan_of(4, 64, 64, 8, 2, "silu", "f16", False, True)
    Y = torch.zeros_like(t["X"])
    five = torch.zeros(5, 64, dtype=torch.float16, device="cuda")
    for call in (lambda: plan.run(five, t["W_router"], t["W_up"], t["W_down"], torch.zeros_like(five)),
                 lambda: plan.run(t["X"], t["W_router"][:7], t["W_up"], t["W_down"], Y),
                 lambda: plan.run(t["X"], t["W_router"], t["W_up"].bfloat16(), t["W_down"], Y),
                 lambda: plan.run(t["X"], t["W_router"], t["W_up"], t["W_down"], Y, torch.zeros(8, 64, dtype=torch.float16, device="cuda"),
                                  torch.zeros(8, 64, dtype=torch.float16, device="cuda")),
                 lambda: plan.run(torch.zeros(4, 67, dtype=torch.float16, device="cuda")[:, :64], t["W_router"], t["W_up"], t["W_down"], Y)):
        with pytest.raises(kt_mlp.KtError) as e:
            call()
        assert e.value.status == kt_mlp.KT_ERR_INVALID
    torch.cuda.synchronize()
    assert plan.status() == kt_mlp.KT_OK


@pytest.mark.parametrize("T,D,F,E,k,act,dtype", [(1, 640, 1280, 8, 2, "geglu", "bf16"), (20, 640, 2560, 16, 2, "geglu", "f16"),
                                                 (64, 256, 520, 12, 4, "gelu_tanh", "bf16")])
def test_new_tokens_through_the_same_workspace(T, D, F, E, k, act, dtype):
    """Runs of changing tokens right behind one another: no block reads a hidden layer or a sum of the
    run before, so every result is that of the run alone, bit for bit."""
    steps = 16
    t = problem(T, D, F, E, k, act, dtype, False, 9)
    xs = [problem(T, D, F, E, k, act, dtype, False, 30 + i)["X"] * (1.0 + i) for i in range(steps)]
    plan = plan_of(T, D, F, E, k, act, dtype, False, True)
    alone = [run(plan, {**t, "X": x})[0] for x in xs]
    check(run(plan, {**t, "X": xs[3]}), reference({**t, "X": xs[3]}, None, k, act, True))
    for _ in range(3):
        again = [torch.full_like(x, float("nan")) for x in xs]
        for x, y in zip(xs, again):
            plan.run(x, t["W_router"], t["W_up"], t["W_down"], y)
        assert plan.status() == kt_mlp.KT_OK
        assert all(torch.equal(a, b) for a, b in zip(alone, again))


def test_the_status_covers_replays_on_any_stream():
    """A graph captured on one stream and replayed on another: the status waits for the replays."""
    t = problem(4, 64, 64, 8, 2, "silu", "f16", False, 10)
    plan = plan_of(4, 64, 64, 8, 2, "silu", "f16", False, True)
    want, _, _ = run(plan, t)
    got = torch.full_like(want, float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(t["X"], t["W_router"], t["W_up"], t["W_down"], got)
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        graph.replay()
        done.record()
    assert plan.status() == kt_mlp.KT_OK
    assert done.query()
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,D,F,E,k,act,dtype", [(1, 640, 1280, 8, 2, "geglu", "bf16"), (9, 256, 4304, 16, 2, "gelu_tanh", "f16"),
                                                 (64, 256, 520, 12, 4, "geglu", "bf16")])
def test_a_wait_that_runs_out_is_reported_and_the_plan_recovers(T, D, F, E, k, act, dtype):
    """The first block waits, for 20 ms, on a barrier that nobody signals; the others give up with it.
    Runs behind it do nothing until the status has been asked."""
    t = problem(T, D, F, E, k, act, dtype, False, 11)
    plan = plan_of(T, D, F, E, k, act, dtype, False, True)
    want, _, _ = run(plan, t)
    got = torch.full_like(want, 7.0)
    args = (t["X"], t["W_router"], t["W_up"], t["W_down"], got)
    kt_ops.kt_moe_debug_stall(plan.handle, True, 20000)
    plan.run(*args)
    kt_ops.kt_moe_debug_stall(plan.handle, False)
    plan.run(*args)
    assert plan.status() == kt_mlp.KT_ERR_TIMEOUT
    assert (got == 7).all()
    assert plan.status() == kt_mlp.KT_OK
    for _ in range(2):
        again, _, _ = run(plan, t)
        assert torch.equal(again, want)


def test_the_status_sees_a_replay_that_ran_out_on_another_stream():
    t = problem(4, 64, 64, 8, 2, "silu", "f16", False, 10)
    plan = plan_of(4, 64, 64, 8, 2, "silu", "f16", False, True)
    want, _, _ = run(plan, t)
    got = torch.full_like(want, 7.0)
    kt_ops.kt_moe_debug_stall(plan.handle, True, 20000)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(t["X"], t["W_router"], t["W_up"], t["W_down"], got)
    kt_ops.kt_moe_debug_stall(plan.handle, False)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        graph.replay()
    assert plan.status() == kt_mlp.KT_ERR_TIMEOUT
    again, _, _ = run(plan, t)
    assert torch.equal(again, want)


def test_one_token_in_place_in_a_wider_row():
    t = problem(1, 64, 136, 8, 2, "silu", "f16", False, 12)
    plan = plan_of(1, 64, 136, 8, 2, "silu", "f16", False, True)
    want, _, _ = run(plan, t, R=t["X"])
    wide = torch.full((1, 96), 7.0, dtype=torch.float16, device="cuda")
    wide[:, :64] = t["X"]
    x = wide[:, :64]
    got, _, _ = run(plan, {**t, "X": x}, R=x, Y=x)
    assert torch.equal(got, want) and (wide[:, 64:] == 7).all()
