"""The operators of a training step and of serving in 8-bit floating point together, as the example runs them."""
import pytest
import torch

from transformer_mlp_gemms_gb300 import kt_ops


pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_mlp_gemms_gb300 import build
    build.build()
    kt_ops.load()


def formula(x, w):
    n = torch.nn.functional.layer_norm(x, x.shape[1:], w["gamma"], w["beta"], 1e-5)
    value, gate = (n @ w["up"].t() + w["b_up"]).chunk(2, 1)
    return (value * 0.5 * gate * torch.special.erfc(-gate / 2.0 ** 0.5)) @ w["down"].t() + w["b_down"]


def test_gradients_of_the_sublayer():
    """Against the formula in 64 bits from the same bf16 parameters.  Between the inputs and a gradient lie at most eight
    roundings to bf16 (the norm, p, h, y, dh, dp, the norm's gradient, the result), each off by 2^-8 of its value at most.
    The matrices are random, so a relative error passes through a product as its operand does, and act and act' change
    by about as much as their argument: 8 * 2^-8 of each result's norm, if the roundings added up plainly."""
    from transformer_mlp_gemms_gb300 import example_train as ex
    M, D, F = 200, 144, 336
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = torch.randn(2, M, D, generator=g, device="cuda").bfloat16().unbind()
    layer = ex.Sublayer(M, D, F, ex.init(D, F, seed=4))
    y = layer.forward(x).clone()
    dx = layer.backward(dy, x)
    leaves = {k: t.double().requires_grad_() for k, t in layer.w.items()}
    xd = x.double().requires_grad_()
    want = formula(xd, leaves)
    want.backward(dy.double())
    for name, got, exact in [("y", y, want.detach()), ("x", dx, xd.grad)] + [(k, layer.grad[k], t.grad) for k, t in leaves.items()]:
        assert ((got.double() - exact).norm() / exact.norm()).item() <= 8 * 2.0 ** -8, name


def test_training_replays_the_step():
    """The graph's steps are the steps: the same parameters and losses, and the layer has the parameters' roundings."""
    from transformer_mlp_gemms_gb300 import example_train as ex
    size = dict(M=136, D=144, F=336, steps=4)
    layer, params, losses = ex.train(**size)
    _, again, eager = ex.train(**size, replay=False)
    first = ex.init(size["D"], size["F"], seed=2)
    for k, p in params.items():
        assert torch.equal(p, again[k]) and p.isfinite().all() and not torch.equal(p, first[k]), k
        assert torch.equal(layer.w[k], p.bfloat16()), k
    assert losses == eager


def test_serving_is_near_the_bf16_sublayer():
    """A rounding to e4m3 is off by up to 2^-4 / m of the value for a mantissa m in [1, 2), uniformly: 2^-4 / sqrt(3) *
    sqrt(1/2) = 0.026 of a vector's norm.  Four of them (two operands of two products) added plainly are 0.104 (0.051 in
    squares)."""
    from transformer_mlp_gemms_gb300 import example_train as ex
    g = torch.Generator(device="cuda").manual_seed(5)
    for M in (3, 200):
        x = torch.randn(M, 288, generator=g, device="cuda").bfloat16()
        layer = ex.Sublayer(M, 288, 656, ex.init(288, 656, seed=6))
        exact = layer.forward(x).float()
        y = ex.serve(x, layer.w)
        assert ((y.float() - exact).norm() / exact.norm()).item() < 0.104
