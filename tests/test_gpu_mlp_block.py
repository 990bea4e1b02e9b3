"""examples/mlp_block.py: the operators chained as a block uses them, against autograd in 64 bits.

Bounds (norm-wise, relative): every tensor on the way is rounded once to f16, 2^-11 of its value
at most; the output passes 4 such roundings (h, y, u and itself), a gradient at most 5 more
(du, dpre, dy, the sum, itself).  Each counts with a factor of about 1 in the norm (weights are
scaled to keep it); 16 roundings are allowed for outputs and 32 for gradients.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from linear_norm_util import act  # noqa: E402

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "mlp_block.py")


def example():
    spec = importlib.util.spec_from_file_location("mlp_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def relative(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("tokens,dim,hidden,activation", [(37, 72, 200, "gelu_tanh"),
                                                          (300, 257, 513, "silu"),
                                                          (1, 64, 96, "gelu")])
def test_block_against_autograd(tokens, dim, hidden, activation):
    block = example().MLPBlock(dim, hidden, activation, torch.float16, seed=3)
    torch.manual_seed(5)
    for p in block.parameters():
        p.add_((0.1 * torch.randn(p.shape, device="cuda")).to(p.dtype) * (p.dim() == 1))
    x, r, dout = (torch.randn((tokens, dim), device="cuda").half() for _ in range(3))
    out, kept = block.forward(x, r)
    dx, grads = block.backward(dout, kept)

    p64 = [p.detach().double().cpu().requires_grad_() for p in block.parameters()]
    x64 = x.double().cpu().requires_grad_()
    norm, up, up_bias, down, down_bias = p64
    h = x64 + r.double().cpu()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5) * norm
    want = act(y @ up.t() + up_bias, activation) @ down.t() + down_bias + h
    want.backward(dout.double().cpu())
    assert relative(out, want.detach()) <= 16 * 2.0 ** -11
    assert relative(dx, x64.grad) <= 32 * 2.0 ** -11
    for got, p in zip(grads, p64):
        assert got.shape == p.shape
        assert relative(got, p.grad) <= 32 * 2.0 ** -11


def test_training_lowers_the_loss_and_serving_agrees():
    m = example()
    block = m.MLPBlock(256, 512)
    torch.manual_seed(6)
    x, r, target = (torch.randn((512, 256), device="cuda").bfloat16() for _ in range(3))
    losses = m.train(block, x, r, target, 10, 0.05)
    assert losses[-1] < 0.9 * losses[0]
    block.prepare_serving()
    full, _ = block.forward(x[:3], r[:3])
    eight = block.serve(x[:3], r[:3])
    # y and W_up rounded to 8 bits: 2^-4 of their values at most, both
    assert relative(eight, full.double().cpu()) <= 2 * 2.0 ** -4
