"""gelu and its slope in the lower tail, relative to their own values.

Bounds.  exp(-v^2 / 2) is 2^x of an fp32 argument of magnitude up to 122 at |v| = 13, which three
roundings (v^2, the product with log2 e, log2 e itself) put off by up to 3 2^-24 of itself, times
ln 2: 2^-16.2 of the result.  The cumulative function beside it adds less than 2^-19.  2^-15
covers both and the products that follow; results below 2^-120 may be cut off by subnormal steps
on the way."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import act, half_step, slope  # noqa: E402

pytestmark = pytest.mark.gpu

TAIL = 2.0 ** -15


def slopes(v, activation, small):
    """act'(v) through the bias gradient of one row (and, `small`, the one-launch pass)."""
    n = v.numel()
    dc = torch.ones((1, n), dtype=v.dtype, device="cuda")
    a = torch.ones((1, 8), dtype=v.dtype, device="cuda")
    b = torch.zeros((8, n), dtype=v.dtype, device="cuda")
    return g.linear_backward(dc, a, b, v[None, :], activation=activation, bias_grad=True,
                             a_grad=small, b_grad=small)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gelus_tail_relative_to_its_value(dtype):
    v = torch.linspace(-12.5, -0.01, 4000, device="cuda").to(dtype)
    one = torch.ones((1, 1), dtype=dtype, device="cuda")
    got = g.linear(one, v[None, :], activation="gelu")[0].double()
    want = act(v.double(), "gelu")
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -120
    bound = (half_step(dtype) * (1 + TAIL) + TAIL) * want.abs() + tiny
    worst = ((got - want).abs() / bound).max().item()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("small", [False, True])
def test_gelus_slope_in_its_tail(small):
    """Below -2 the slope's two terms differ by a factor of 4 at least: no cancellation counts."""
    v = torch.linspace(-12.5, -2.0, 4000, device="cuda").bfloat16()
    got = slopes(v, "gelu", small)[2].double()
    want = slope(v.double(), "gelu")
    bound = (half_step(torch.bfloat16) * (1 + 2 * TAIL) + 2 * TAIL) * want.abs() + 2.0 ** -120
    worst = ((got - want).abs() / bound).max().item()
    assert worst <= 1.0, worst
