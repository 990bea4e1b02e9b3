"""Tensors that autograd follows: the linear layer's and the norm's functions take no part in it,
and say so."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402

pytestmark = pytest.mark.gpu


def ones(*shape, dtype=torch.float16):
    return torch.ones(shape, device="cuda").to(dtype)


def grad(t):
    return t.requires_grad_()


@pytest.mark.parametrize("call", [
    lambda: g.linear(grad(ones(4, 8)), ones(8, 16)),
    lambda: g.linear(ones(4, 8), grad(ones(16, 8)).t()),
    lambda: g.linear(ones(4, 8), ones(8, 16), grad(ones(16))),
    lambda: g.linear(ones(4, 8), ones(8, 16), None, grad(ones(4, 16))),
    lambda: g.linear(ones(4, 8), ones(8, 16), out=grad(ones(4, 16))),
    lambda: g.linear_backward(ones(4, 16), grad(ones(4, 8)), ones(8, 16)),
    lambda: g.linear_backward(grad(ones(4, 16)), ones(4, 8), ones(8, 16)),
    lambda: g.rms_norm(grad(ones(4, 8)), ones(8)),
    lambda: g.rms_norm(ones(4, 8), grad(ones(8))),
    lambda: g.rms_norm(ones(4, 8), ones(8), grad(ones(4, 8))),
    lambda: g.rms_norm_backward(ones(4, 8), ones(4, 8), grad(ones(8)),
                                torch.ones(4, device="cuda"))])
def test_a_gradient_is_not_lost_in_silence(call):
    with pytest.raises(ValueError, match="requires grad"):
        call()
    with torch.no_grad():
        call()
    with torch.inference_mode():
        call()


def test_a_forward_mode_tangent_is_not_lost_in_silence():
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        x = fwd.make_dual(ones(4, 8), ones(4, 8))
        with pytest.raises(ValueError, match="requires grad"):
            g.linear(x, ones(8, 16))


def test_an_autograd_function_around_the_calls():
    """The way to have gradients: forward and backward of a torch.autograd.Function."""
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, b):
            ctx.save_for_backward(a, b)
            return g.linear(a, b)

        @staticmethod
        def backward(ctx, dc):
            return g.linear_backward(dc.contiguous(), *ctx.saved_tensors)[:2]

    a, w = grad(ones(4, 8)), grad(ones(16, 8))
    Linear.apply(a, w.t()).sum().backward()
    assert bool((a.grad == 16).all()) and bool((w.grad == 4).all())
