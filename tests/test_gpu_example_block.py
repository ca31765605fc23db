"""The operators together, as the example runs them."""
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


def test_decoding_replays_the_block():
    from transformer_mlp_gemms_gb300 import example_block as ex
    one, _ = ex.decode(tokens=3, D=128, F=192, steps=1)
    two, _ = ex.decode(tokens=3, D=128, F=192, steps=2)
    again, _ = ex.decode(tokens=3, D=128, F=192, steps=2)
    assert torch.equal(two, again) and not torch.equal(one, two) and two.isfinite().all()


def test_quantised_mlp_is_near_the_fp16_one():
    """Rounding to integers of a row's 1/127: an error of at most 0.5/127 of the row's largest
    value, uniform, so sqrt(1/12)/127 = 0.0023 of it; a normal row's largest value is 3.2 to 3.6
    times its root mean square at these lengths, after the activation at most 7 times.  Four
    roundings (two operands of two products) add up in squares: below 2 * 0.0081 + 0.0023 * 7 = 0.033
    even if added plainly."""
    from transformer_mlp_gemms_gb300 import example_block as ex
    y, exact = ex.quantised_mlp(M=100, D=320, F=1008)
    assert ((y.float() - exact.float()).norm() / exact.float().norm()).item() < 0.033


def test_training_a_norm_converges():
    """Per column the loss is quadratic with a curvature of about 1: steps of 0.5 halve the error
    each time, down to bf16's rounding of y (2^-9 of values around 1, squared 4e-6, on both sides,
    and of gamma and beta)."""
    from transformer_mlp_gemms_gb300 import example_block as ex
    losses = ex.train_norm(M=256, D=96, steps=40)
    assert losses[10] < losses[0] * 0.25 ** 5 + 1e-4 and losses[-1] < 1e-4
