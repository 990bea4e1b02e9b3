"""Checkpoints of empty batches and of layers without inputs: made by the linear layer, and read by its
backward pass with every activation that recomputes the layer's input."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from test_gpu_mlp_block import example  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("a_activation", ACTS)
@pytest.mark.parametrize("activation", ["none", "silu"])
@pytest.mark.parametrize("m,n,k", [(0, 14, 10), (6, 0, 10), (6, 14, 0), (0, 14, 0), (0, 0, 10)])
def test_backward(m, n, k, activation, a_activation, dt):
    def ones(*shape):
        return torch.ones(shape, dtype=dt, device="cuda")

    print(f"empty {m}x{n}x{k} {activation} {a_activation}", flush=True)
    da, db, dbias = g.linear_backward(ones(m, n), g.pack8(ones(m, k)), ones(k, n), g.pack8(ones(m, n)),
                                      activation=activation, a_activation=a_activation,
                                      bias_grad=True)
    assert da.shape == (m, k) and db.shape == (k, n) and dbias.shape == (n,)
    if n == 0:
        assert not da.any()
    if m == 0:
        assert not db.any() and not dbias.any()


def test_block_on_no_tokens():
    block = example().MLPBlock(64, 96, norm="layer", keep8=True)
    x = torch.ones((0, 64), dtype=torch.bfloat16, device="cuda")
    out, kept = block.forward(x, x)
    dx, grads = block.backward(out, kept)
    assert out.shape == dx.shape == (0, 64)
    for grad, p in zip(grads, block.parameters()):
        assert grad.shape == p.shape and not grad.any()


@pytest.mark.parametrize("ty", [torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("m,n,k", [(5, 45, 0), (40, 77, 0), (300, 7, 0), (0, 45, 16), (5, 0, 16)])
def test_linear(m, n, k, ty):
    """Without inputs the value before the activation is the bias."""
    dt = ty if ty.itemsize == 2 else torch.float16
    a, w = (torch.ones((x, k), device="cuda").to(ty) for x in (m, n))
    bias = (torch.arange(n, device="cuda") % 9).to(dt)
    print(f"empty linear {m}x{n}x{k} {ty}", flush=True)
    out, p = g.linear(a, w.t(), bias, activation="relu", out_dtype=dt, pack_pre=True)
    assert out.shape == p.values.shape == (m, n) and p.scale.shape == (m, -(-n // 32))
    if k == 0:
        assert torch.equal(out, bias.expand(m, n))
        assert torch.equal(g.unpack8(p, dtype=dt), bias.expand(m, n))
