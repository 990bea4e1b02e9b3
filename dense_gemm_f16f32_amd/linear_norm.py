"""The linear layer with its epilogue, the root-mean-square norm, and their backward passes, for
torch tensors (see include/linear_norm.h for the formulas and contracts).

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
                     "rms_norm_backward"):
            f = getattr(L, name)
            f.argtypes, f.restype = [ctypes.c_char_p], ctypes.c_int
        for name in ("linear_forward_workspace", "linear_backward_workspace",
                     "rms_norm_backward_workspace"):
            f = getattr(L, name)
            f.argtypes, f.restype = [ctypes.c_char_p], ctypes.c_int64
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


def linear(a, b, bias=None, residual=None, *, activation="none", scale_a=None, scale_b=None,
           out_dtype=None, with_pre=False, out=None, stream=None):
    """act(a @ b + bias) + residual on the GPU: fp32 sums, one rounding (8-bit operands with more
    than 16 rows and k above 512: the matrix instruction's own sums, off by up to 2^-17 of the sum
    of the products' magnitudes at k = 1000).

    a (m, k) and b (k, n): float16 or bfloat16, each row- or column-major with any leading
    dimension (a weight stored (n, k) is passed as `w.t()`); or float8_e4m3fn, k-contiguous (a
    row-major, b column-major) with 16-byte aligned rows, and `scale_a` (m,) and `scale_b` (n,)
    float32 factors of the rows and columns (1 if not given).  bias (n,), residual (m, n): of
    the output's type, which is the operands' (8-bit operands: `out_dtype`, bfloat16 if not
    given).  activation: none, relu, gelu, gelu_tanh or silu.  Returns the (m, n) result, or
    (result, pre) with `with_pre`, where pre is the value before the activation, which
    linear_backward needs.  `out` may be the residual's own tensor.
    """
    f = (_native or native()).linear
    if stream is None:
        return f(a, b, bias, residual, activation, scale_a, scale_b, out_dtype, with_pre, out)
    args = (a, b, bias, residual, activation, scale_a, scale_b, out_dtype, with_pre, out)
    return _on(stream, f, args, (a, b, bias, residual, scale_a, scale_b, out))


def linear_backward(dc, a, b, pre=None, *, activation="none", bias_grad=False, a_grad=True,
                    b_grad=True, stream=None):
    """(da, db, dbias): gradients of linear's a, b and bias (None where not asked for).

    dc (m, n) is the gradient of linear's result; that of its residual is dc itself.  pre (m, n)
    is linear's value before the activation (not needed for "none").  All of one 16-bit type;
    dc and pre contiguous along n, a and b as in linear.  db has b's storage order.

    dc act'(pre) is rounded to that type before it enters the two products, which take 16-bit
    operands: da and db are off by about 0.0023 (bfloat16) or 0.0003 (float16) of their norms,
    where the rounding of the results alone would leave 0.0017 and 0.0002.  dbias sums the
    unrounded values.
    """
    f = (_native or native()).linear_backward
    if stream is None:
        return f(dc, a, b, pre, activation, bias_grad, a_grad, b_grad)
    return _on(stream, f, (dc, a, b, pre, activation, bias_grad, a_grad, b_grad),
               (dc, a, b, pre))


def rms_norm(x, weight, residual=None, *, eps=1e-5, out_dtype=None, with_rstd=False,
             stream=None):
    """RMSNormResult of h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.

    x, residual (rows, dim) and weight (dim,): one 16-bit type, rows contiguous, any row stride.
    y has that type, or with out_dtype=torch.float8_e4m3fn it is y / scale in 8 bits, with one
    float32 scale a row, laid out as linear's 8-bit operand.  h is rounded to x's type; the norm
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
