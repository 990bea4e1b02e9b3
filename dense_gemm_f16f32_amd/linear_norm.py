"""The linear layer with its epilogue, the root-mean-square norm, the layer norm, their backward
passes, and activations in 8 bits, for torch tensors (see include/linear_norm.h for the formulas and
contracts).

Every step of the computation runs in the HIP kernels of liblinear_norm.so.  The functions here
go through the compiled binding csrc/torch_binding.cpp, which checks the tensors, allocates
results and workspace with torch on the stream the kernels run on, and calls the library.
With `stream` a call runs on that stream; the caller orders it after the work that makes its
operands, and the work that uses its results after it, as with any torch stream.  Operands may be
temporaries.  Errors found by the library raise `GemmError` with its code; what it cannot see
(dtypes, devices, shapes) raises ValueError.  The functions keep no state and take no part in autograd
(the *_backward functions are the gradients): an operand that requires grad is refused, outside
torch.no_grad() and the forward and backward of a torch.autograd.Function.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "liblinear_norm.so")
BINDING_PATH = os.path.join(PKG, "_linear_norm.so")

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")

_lib = None
_native = None


def lib() -> ctypes.CDLL:
    """The library's C entry points (each takes the address of its argument structure); raises
    if liblinear_norm.so has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(or python dense_gemm_f16f32_amd/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        for name in ("linear_forward", "linear_backward", "rms_norm_forward",
                     "rms_norm_backward", "layer_norm_forward", "layer_norm_backward",
                     "quantize_rows", "pack8", "unpack8"):
            f = getattr(L, name)
            f.argtypes, f.restype = [ctypes.c_char_p], ctypes.c_int
        for name in ("linear_forward_workspace", "linear_backward_workspace",
                     "rms_norm_backward_workspace", "layer_norm_backward_workspace"):
            f = getattr(L, name)
            f.argtypes, f.restype = [ctypes.c_char_p], ctypes.c_int64
        for name in ("linear_forward_packed", "linear_backward_packed"):
            f, w = getattr(L, name), getattr(L, name + "_workspace")
            f.argtypes = w.argtypes = [ctypes.c_char_p, ctypes.c_char_p]
            f.restype, w.restype = ctypes.c_int, ctypes.c_int64
        _lib = L
    return _lib


def native():
    """The compiled binding; raises if it has not been built."""
    global _native
    if _native is None:
        import importlib.util

        import torch  # noqa: F401  (the binding links against it)
        for path in (LIB_PATH, BINDING_PATH):
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                                   "(or python dense_gemm_f16f32_amd/build.py)")
        spec = importlib.util.spec_from_file_location("_linear_norm", BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native = module
    return _native


def _on(stream, f, args, tensors):
    """f(*args) on `stream` instead of torch's current one.  The tensors among args stay
    untouched until `stream` has passed the call: torch gives memory that is freed before that
    to no other work."""
    import torch
    t = tensors[0]
    if isinstance(t, torch.Tensor) and t.is_cuda and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the operands on {t.device}")
    with torch.cuda.stream(stream):
        result = f(*args)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return result


class RMSNormResult(NamedTuple):
    y: object       # the normalised rows
    h: object       # x + residual (x itself without a residual)
    rstd: object    # float32, one a row; None unless asked for
    scale: object   # float32, one a row; None unless y is in 8 bits


class LayerNormResult(NamedTuple):
    y: object       # the normalised rows
    h: object       # x + residual (x itself without a residual)
    mean: object    # float32, one a row; None unless asked for
    rstd: object    # float32, one a row; None unless asked for
    scale: object   # float32, one a row; None unless y is in 8 bits


class QuantizedRows(NamedTuple):
    values: object  # (rows, dim) int8 or float8_e4m3fn, laid out as linear's 8-bit operand
    scale: object   # float32, one a row


class Packed8(NamedTuple):
    """A (rows, dim) matrix in 8 bits: values[i, j] * scale[i, j // 32]."""
    values: object  # (rows, dim) int8
    scale: object   # (rows, ceil(dim / 32)) float8_e8m0fnu: powers of two


def linear(a, b, bias=None, residual=None, *, activation="none", scale_a=None, scale_b=None,
           out_dtype=None, with_pre=False, pack_pre=False, out=None, stream=None):
    """act(a @ b + bias) + residual on the GPU: fp32 sums, one rounding (float8_e4m3fn operands with
    more than 16 rows and k above 512: the matrix instruction's own sums, off by up to 2^-17 of the
    sum of the products' magnitudes at k = 1000; int8 operands: exact 32-bit integer sums).

    a (m, k) and b (k, n): float16 or bfloat16, each row- or column-major with any leading
    dimension (a weight stored (n, k) is passed as `w.t()`); or float8_e4m3fn or int8 (k up to
    131071), k-contiguous (a row-major, b column-major) with 16-byte aligned rows, and `scale_a`
    (m,) and `scale_b` (n,) float32 factors of the rows and columns (1 if not given).  bias (n,),
    residual (m, n): of the output's type, which is the operands' (8-bit operands: `out_dtype`,
    bfloat16 if not given).  activation: none, relu, gelu, gelu_tanh or silu.  Returns the (m, n) result, or
    (result, pre) with `with_pre`, where pre is the value before the activation, which
    linear_backward needs; with `pack_pre` pre is a Packed8, of half the size, made of the unrounded
    values (with relu, whose slope goes by the sign, a positive value is 1 scale at least).  `out` may be
    the residual's own tensor.
    """
    f = (_native or native()).linear
    packed = Packed8 if pack_pre else None
    if stream is None:
        return f(a, b, bias, residual, activation, scale_a, scale_b, out_dtype, with_pre, out,
                 packed)
    args = (a, b, bias, residual, activation, scale_a, scale_b, out_dtype, with_pre, out, packed)
    return _on(stream, f, args, (a, b, bias, residual, scale_a, scale_b, out))


def linear_backward(dc, a, b, pre=None, *, activation="none", bias_grad=False, a_grad=True,
                    b_grad=True, a_activation="none", stream=None):
    """(da, db, dbias): gradients of linear's a, b and bias (None where not asked for).

    dc (m, n) is the gradient of linear's result; that of its residual is dc itself.  pre (m, n)
    is linear's value before the activation (not needed for "none").  All of one 16-bit type;
    dc and pre contiguous along n, a and b as in linear.  db has b's storage order.  a, pre or both
    may be Packed8, as pack8 and linear's pack_pre make them.  With a_activation, a Packed8 `a` holds
    the values before that activation, from which the layer's input is computed again (rounded to
    the 16-bit type, as the layer that made it rounded it); da is the gradient of that input.

    dc act'(pre) is rounded to that type before it enters the two products, which take 16-bit
    operands: da and db are off by about 0.0023 (bfloat16) or 0.0003 (float16) of their norms,
    where the rounding of the results alone would leave 0.0017 and 0.0002.  dbias sums the
    unrounded values.
    """
    f = (_native or native()).linear_backward
    a_scale = pre_scale = None
    if isinstance(a, Packed8):
        a, a_scale = a
    if isinstance(pre, Packed8):
        pre, pre_scale = pre
    args = (dc, a, b, pre, activation, bias_grad, a_grad, b_grad, a_scale, pre_scale, a_activation)
    if stream is None:
        return f(*args)
    return _on(stream, f, args, (dc, a, b, pre, a_scale, pre_scale))


def rms_norm(x, weight, residual=None, *, eps=1e-5, out_dtype=None, with_rstd=False,
             stream=None):
    """RMSNormResult of h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.

    x, residual (rows, dim) and weight (dim,): one 16-bit type, rows contiguous, any row stride.
    y has that type, or with out_dtype=torch.float8_e4m3fn or torch.int8 it is y / scale in 8 bits,
    with one float32 scale a row, laid out as linear's 8-bit operand.  h is rounded to x's type; the norm
    is taken of the unrounded sum.  `with_rstd` also returns 1 / sqrt(mean(h^2) + eps), which
    rms_norm_backward needs.
    """
    f = (_native or native()).rms_norm
    if stream is None:
        return f(x, weight, residual, eps, out_dtype, with_rstd, RMSNormResult)
    return _on(stream, f, (x, weight, residual, eps, out_dtype, with_rstd, RMSNormResult),
               (x, weight, residual))


def rms_norm_backward(dy, h, weight, rstd, *, dh=None, weight_grad=True, stream=None):
    """(dx, dweight) of rms_norm: dx is the gradient of x and of the residual alike.

    dy (rows, dim): gradient of y; h and rstd as rms_norm returned them; dh: the gradient that
    reaches h by another way (the residual stream), added to dx.
    """
    f = (_native or native()).rms_norm_backward
    if stream is None:
        return f(dy, h, weight, rstd, dh, weight_grad)
    return _on(stream, f, (dy, h, weight, rstd, dh, weight_grad), (dy, h, weight, rstd, dh))


def layer_norm(x, weight, bias=None, residual=None, *, eps=1e-5, out_dtype=None, with_stats=False,
               stream=None):
    """LayerNormResult of h = x + residual, y = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias.

    x, residual (rows, dim), weight and bias (dim,): one 16-bit type, rows contiguous, any row
    stride.  var is the mean of the squares of h - mean(h).  y has that type, or with out_dtype=
    torch.float8_e4m3fn or torch.int8 it is y / scale in 8 bits, with one float32 scale a row, laid
    out as linear's 8-bit operand.  h is rounded to x's type; the norm is taken of the unrounded sum.
    `with_stats` also returns mean(h) and 1 / sqrt(var(h) + eps), which layer_norm_backward needs.
    """
    f = (_native or native()).layer_norm
    if stream is None:
        return f(x, weight, bias, residual, eps, out_dtype, with_stats, LayerNormResult)
    return _on(stream, f, (x, weight, bias, residual, eps, out_dtype, with_stats, LayerNormResult),
               (x, weight, bias, residual))


def layer_norm_backward(dy, h, weight, mean, rstd, *, dh=None, weight_grad=True, bias_grad=True,
                        stream=None):
    """(dx, dweight, dbias) of layer_norm: dx is the gradient of x and of the residual alike.

    dy (rows, dim): gradient of y; h, mean and rstd as layer_norm returned them; dh: the gradient
    that reaches h by another way (the residual stream), added to dx.
    """
    f = (_native or native()).layer_norm_backward
    if stream is None:
        return f(dy, h, weight, mean, rstd, dh, weight_grad, bias_grad)
    return _on(stream, f, (dy, h, weight, mean, rstd, dh, weight_grad, bias_grad),
               (dy, h, weight, mean, rstd, dh))


def quantize_rows(x, *, dtype=None, stream=None):
    """QuantizedRows of x (rows, dim) of a 16-bit type, rows contiguous: 8-bit values and one scale
    a row, operand and scale_a of linear.

    dtype int8 (if not given): scale = max |x| / 127 and values = x / scale to the nearest integer,
    ties to even; float8_e4m3fn: with 448 in the place of 127.  A row of zeros has scale 1.  An int8
    row with a NaN or an infinity has scale NaN.
    """
    f = (_native or native()).quantize_rows
    if stream is None:
        return f(x, dtype, QuantizedRows)
    return _on(stream, f, (x, dtype, QuantizedRows), (x,))


def pack8(x, *, stream=None):
    """Packed8 of x (rows, dim) of a 16-bit type, rows contiguous: an activation kept in 8 bits for
    linear_backward.

    Each 32 neighbours of a row share a power of two, by which the largest of them lies in [64, 128);
    values are rounded to the nearest integer, ties to even, and are at most 127 in magnitude, so
    they are off by at most half a step (a whole one above 127.5 steps).  Positive values of up to
    half a step become 0, where relu's slope is 0: for its backward pass keep linear's pack_pre,
    which leaves them positive.  Scales are at least 2^-24 (float16) or 2^-120 (bfloat16): values
    times scales are numbers of x's type.  A block that holds a NaN or an infinity has scale NaN,
    and linear_backward has NaN for its gradients.
    """
    f = (_native or native()).pack8
    return f(x, Packed8) if stream is None else _on(stream, f, (x, Packed8), (x,))


def unpack8(packed, *, dtype=None, activation="none", stream=None):
    """act(values * scale) of a Packed8, in `dtype` (bfloat16 if not given, or float16)."""
    if not isinstance(packed, Packed8):
        raise TypeError("packed must be a Packed8")
    f = (_native or native()).unpack8
    args = (packed.values, packed.scale, dtype, activation)
    return f(*args) if stream is None else _on(stream, f, args, packed)
