"""A transformer block's MLP, trained and then served, on the linear layer's and norm's operators.

    h = x + residual;  y = rms_norm(h);  out = act(y W_up^T + b_up) W_down^T + b_down + h

Training keeps what the backward pass needs (h, rstd, y, the pre-activation, the activation) and
chains linear_backward and rms_norm_backward; the weights are updated by plain SGD.  Serving
quantises the up-projection once, norms each token into 8 bits and reads the 8-bit weights.

    python examples/mlp_block.py [--dim 1024 --hidden 4096 --tokens 2048 --steps 40 --rate 0.002]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_f16f32_amd as g  # noqa: E402


class MLPBlock:
    """Parameters as (out, in) matrices; every method runs on torch's current stream."""

    def __init__(self, dim, hidden, activation="gelu_tanh", dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=gen, device="cuda") * cols ** -0.5
            return w.to(dtype)

        self.activation = activation
        self.norm = torch.ones(dim, dtype=dtype, device="cuda")
        self.up, self.up_bias = weight(hidden, dim), torch.zeros(hidden, dtype=dtype, device="cuda")
        self.down, self.down_bias = weight(dim, hidden), torch.zeros(dim, dtype=dtype,
                                                                     device="cuda")
        self.up8 = self.up8_scale = None

    def parameters(self):
        return [self.norm, self.up, self.up_bias, self.down, self.down_bias]

    def forward(self, x, residual):
        n = g.rms_norm(x, self.norm, residual, with_rstd=True)
        u, pre = g.linear(n.y, self.up.t(), self.up_bias, activation=self.activation,
                          with_pre=True)
        out = g.linear(u, self.down.t(), self.down_bias, n.h)
        return out, (n, pre, u)

    def backward(self, dout, kept):
        """(gradient of x and of the residual, gradients in parameters() order)."""
        n, pre, u = kept
        du, d_down, d_down_bias = g.linear_backward(dout, u, self.down.t(), bias_grad=True)
        dy, d_up, d_up_bias = g.linear_backward(du, n.y, self.up.t(), pre,
                                                activation=self.activation, bias_grad=True)
        # dout reaches h directly too, as the residual of the down-projection
        dx, d_norm = g.rms_norm_backward(dy, n.h, self.norm, n.rstd, dh=dout)
        return dx, [d_norm, d_up.t(), d_up_bias, d_down.t(), d_down_bias]

    def prepare_serving(self):
        """The up-projection in 8 bits with a scale an output, rows on 16-byte boundaries."""
        w = self.up.float()
        rows, cols = w.shape
        amax = w.abs().amax(1)
        self.up8_scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        buf = torch.zeros((rows, -(-cols // 16) * 16), dtype=torch.float8_e4m3fn, device="cuda")
        buf[:, :cols] = (w / self.up8_scale[:, None]).to(torch.float8_e4m3fn)
        self.up8 = buf[:, :cols]

    def serve(self, x, residual):
        n = g.rms_norm(x, self.norm, residual, out_dtype=torch.float8_e4m3fn)
        u = g.linear(n.y, self.up8.t(), self.up_bias, activation=self.activation,
                     scale_a=n.scale, scale_b=self.up8_scale, out_dtype=x.dtype)
        return g.linear(u, self.down.t(), self.down_bias, n.h)


def train(block, x, residual, target, steps, rate):
    """Mean squared error to `target`, by SGD; returns the losses."""
    losses = []
    for _ in range(steps):
        out, kept = block.forward(x, residual)
        error = out.float() - target.float()
        losses.append(error.square().mean())
        dout = (error * (2.0 / error.shape[0])).to(out.dtype)
        for p, d in zip(block.parameters(), block.backward(dout, kept)[1]):
            p.sub_((rate * d.float()).to(p.dtype))
    return [v.item() for v in losses]


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("--dim", 1024), ("--hidden", 4096), ("--tokens", 2048),
                        ("--steps", 40)):
        ap.add_argument(name, type=int, default=value)
    ap.add_argument("--rate", type=float, default=0.002)
    a = ap.parse_args()
    torch.manual_seed(1)
    x, residual, target = (torch.randn((a.tokens, a.dim), device="cuda").bfloat16()
                           for _ in range(3))
    block = MLPBlock(a.dim, a.hidden)
    losses = train(block, x, residual, target, a.steps, a.rate)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    block.prepare_serving()
    full, _ = block.forward(x[:1], residual[:1])
    eight = block.serve(x[:1], residual[:1])
    print(f"one token, 8-bit against 16-bit: relative difference "
          f"{((eight - full).float().norm() / full.float().norm()).item():.4f}")
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(200):
        block.serve(x[:1], residual[:1])
    torch.cuda.synchronize()
    print(f"one token served: {(time.perf_counter() - start) / 200 * 1e6:.1f} us")


if __name__ == "__main__":
    main()
