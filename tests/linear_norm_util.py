"""The linear layer's and the norm's operators in 64 bits, and the bounds that the kernels'
results have to meet (shared by the GPU tests).

Bounds.  A result of type t is off by at most half a step, finfo(t).eps / 2 of its value, from
the fp32 value that is rounded.  That value's own error: a sum of K products in fp32, in any
order and with products and partial sums truncated rather than rounded, is off by at most
(K + 8) 2^-23 times the sum of the magnitudes; activations and their slopes, of magnitude up to
1.13 |v| and 1.13, are computed to 2^-20 (the erfc formula's 1.5e-7, a few fp32 roundings of
exp and reciprocal); each further fp32 operation adds 2^-23 of its operands.  fp16 results below
2^-14 have steps of 2^-24.
"""
import math

import torch

F32 = 2.0 ** -23


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the smallest step of a type."""
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133,
            torch.float8_e4m3fn: 2.0 ** -10}[t]


def phi(v):
    return torch.special.erfc(v / -math.sqrt(2.0)) / 2


def act(v, name):
    if name == "relu":
        return v.clamp(min=0)
    if name == "gelu":
        return v * phi(v)
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def slope(v, name):
    """act's derivative (relu: 0 at 0)."""
    if name == "none":
        return torch.ones_like(v)
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "gelu":
        return phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        p = torch.sigmoid(v)
        return p + v * p * (1 - p)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def mm(a, b):
    return torch.mm(a.contiguous(), b.contiguous())


def linear64(a, b, bias=None, residual=None, activation="none", scale_a=None, scale_b=None):
    """(out, pre, bound of the fp32 pre, bound of the fp32 out)."""
    a, b = a.double(), b.double()
    if scale_a is not None:
        a = a * scale_a.double()[:, None]
    if scale_b is not None:
        b = b * scale_b.double()[None, :]
    v, mag = mm(a, b), mm(a.abs(), b.abs())
    err = (a.shape[1] + 8) * F32 * mag
    if bias is not None:
        v = v + bias.double()
        err = err + F32 * (bias.double().abs() + mag)
    out = act(v, activation)
    oerr = 1.13 * err
    if activation not in ("none", "relu"):
        oerr = oerr + 2.0 ** -20 * v.abs()
    if residual is not None:
        out = out + residual.double()
        oerr = oerr + F32 * (residual.double().abs() + out.abs())
    return out, v, err, oerr


def assert_close(got, want, err, what=""):
    """|got - want| <= half a step of got's type + err, element by element."""
    got64 = got.double()
    assert bool(torch.isfinite(got64).all()), f"{what}: not finite"
    bound = half_step(got.dtype) * (want.abs() + err) + err + tiny(got.dtype)
    worst = ((got64 - want).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def strided(t, pad=0, offset=0, fill=float("nan")):
    """A copy of t (2-D, stored as it is: row- or column-major) with `pad` extra elements a
    stored row and `offset` elements before the first; what lies between holds `fill`."""
    col = t.stride(0) == 1 and t.stride(1) != 1
    s = t.t() if col else t
    rows, cols = s.shape
    buf = torch.full((offset + rows * (cols + pad) + 8,), fill, device=t.device).to(t.dtype)
    view = torch.as_strided(buf, (rows, cols), (cols + pad, 1), offset)
    view.copy_(s)
    return view.t() if col else view


def e4m3_rows(v):
    """v in 8 bits with a scale a row, its rows 16-byte aligned, NaN in the padding."""
    amax = v.abs().amax(1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    rows, cols = v.shape
    buf = torch.full((rows, -(-cols // 16) * 16), float("nan"), device=v.device).to(
        torch.float8_e4m3fn)
    buf[:, :cols] = (v / scale[:, None]).to(torch.float8_e4m3fn)
    return buf[:, :cols], scale
