"""examples/mlp_block.py with the layer norm, 8-bit checkpoints and int8 serving: the operators chained
as a block uses them, against autograd in 64 bits.

Bounds (norm-wise, relative): roundings to f16 as in test_gpu_mlp_block.py, 16 of 2^-11 for outputs
and 32 for gradients.  A checkpoint's half step is at most 2^-7 of its block's largest magnitude (of 32
normal values below 4 of their deviations) and uniform: 4 2^-7 / sqrt(3) of the norm of the value
kept.  y enters d_up with a factor of 1; the pre-activation enters all gradients through the slope and
the recomputed activation, whose own slopes are below 1.2: twice that is allowed.  Serving rounds y, u
and the weights to int8, half a step 2^-8 of a row's largest magnitude, at most 6 deviations of a
normal row here: 6 2^-8 / sqrt(3) each, four of them."""
import pytest

torch = pytest.importorskip("torch")

from linear_norm_util import act  # noqa: E402
from test_gpu_mlp_block import example, relative  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("tokens,dim,hidden,activation", [(37, 72, 200, "gelu_tanh"),
                                                          (300, 257, 513, "silu"),
                                                          (1, 64, 96, "gelu")])
def test_block_against_autograd(tokens, dim, hidden, activation, norm, keep8):
    block = example().MLPBlock(dim, hidden, activation, torch.float16, 3, norm, keep8)
    torch.manual_seed(5)
    for p in block.parameters():
        p.add_((0.1 * torch.randn(p.shape, device="cuda")).to(p.dtype) * (p.dim() == 1))
    x, r, dout = (torch.randn((tokens, dim), device="cuda").half() for _ in range(3))
    out, kept = block.forward(x, r)
    dx, grads = block.backward(dout, kept)

    p64 = [p.detach().double().cpu().requires_grad_() for p in block.parameters()]
    x64 = x.double().cpu().requires_grad_()
    weight, up, up_bias, down, down_bias = p64[:5]
    h = x64 + r.double().cpu()
    if norm == "layer":
        c = h - h.mean(1, keepdim=True)
        y = c / torch.sqrt(c.square().mean(1, keepdim=True) + 1e-5) * weight + p64[5]
    else:
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5) * weight
    want = act(y @ up.t() + up_bias, activation) @ down.t() + down_bias + h
    want.backward(dout.double().cpu())
    more = 2 * 4 * 2.0 ** -7 / 3 ** 0.5 if keep8 else 0.0
    assert relative(out, want.detach()) <= 16 * 2.0 ** -11
    assert relative(dx, x64.grad) <= 32 * 2.0 ** -11 + more
    assert len(grads) == len(p64)
    for got, p in zip(grads, p64):
        assert got.shape == p.shape
        assert relative(got, p.grad) <= 32 * 2.0 ** -11 + more


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_int8_serving(norm):
    block = example().MLPBlock(256, 512, norm=norm)
    torch.manual_seed(6)
    for tokens in (1, 5, 40):
        x, r = (torch.randn((tokens, 256), device="cuda").bfloat16() for _ in range(2))
        block.prepare_serving(int8=True)
        full, _ = block.forward(x, r)
        eight = block.serve(x, r)
        assert relative(eight, full.double().cpu()) <= 4 * 6 * 2.0 ** -8 / 3 ** 0.5


def test_training_with_checkpoints_runs():
    m = example()
    block = m.MLPBlock(128, 256, norm="layer", keep8=True)
    x, r, target = (torch.randn((64, 128), device="cuda").bfloat16() for _ in range(3))
    losses = m.train(block, x, r, target, 3, 0.01)
    assert len(losses) == 3 and all(v == v for v in losses)
