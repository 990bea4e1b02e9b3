"""Activations and their slopes towards the ends of the number range: at pre-activations whose
square overflows fp32."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402

pytestmark = pytest.mark.gpu


def slopes(v, activation, small):
    """act'(v) through the bias gradient of one row (and, `small`, the one-launch pass)."""
    n = v.numel()
    dc = torch.ones((1, n), dtype=v.dtype, device="cuda")
    a = torch.ones((1, 8), dtype=v.dtype, device="cuda")
    b = torch.zeros((8, n), dtype=v.dtype, device="cuda")
    return g.linear_backward(dc, a, b, v[None, :], activation=activation, bias_grad=True,
                             a_grad=small, b_grad=small)


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("activation", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_at_large_values(activation, small):
    """1 above, 0 below, for every finite value; the gradients beside them stay finite."""
    top = torch.finfo(torch.bfloat16).max
    v = torch.tensor([1e3, 1e10, 1.8e19, 2e19, 5e19, 1e20, 1e30, 3e38, top], device="cuda")
    v = torch.cat([v, -v]).bfloat16()
    da, db, got = slopes(v, activation, small)
    want = (v > 0).bfloat16()
    assert torch.equal(got, want), got
    if small:
        assert torch.equal(db, want.expand(8, -1)) and not da.any()


@pytest.mark.parametrize("activation", ["gelu_tanh", "gelu", "silu", "relu"])
def test_values_at_large_values(activation):
    v = torch.tensor([1e3, 1.8e19, 1e20, 3e38, -1e3, -1.8e19, -1e20, -3e38], device="cuda").bfloat16()
    one = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda")
    got = g.linear(one, v[None, :], activation=activation)
    assert torch.equal(got[0], v.clamp(min=0))
