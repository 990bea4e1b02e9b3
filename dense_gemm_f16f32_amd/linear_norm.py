"""Python binding of liblinear_norm.so: the linear layer with its epilogue, the root-mean-square
norm, and their backward passes (see include/linear_norm.h for the formulas and contracts).

Every step of the computation runs in the library's HIP kernels; torch supplies device memory
and streams.  Results, and the workspace a call needs, are allocated by torch on the stream the
kernels run on.  Errors found by the library raise `GemmError` with its code; what it cannot see
(dtypes, devices, shapes) raises ValueError.  The functions work on plain tensors and keep no
state; they do not take part in autograd (the *_backward functions are the gradients).
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

import dense_gemm_f16f32_amd as _pkg

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblinear_norm.so")

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_lib = None
_dtypes = None   # torch dtype -> LINEAR_NORM_* code

# The argument structures are arrays of 8-byte fields (linear_norm.h).
_FORWARD = struct.Struct("24q")
_BACKWARD = struct.Struct("24q")
_NORM = struct.Struct("15qdq")
_NORM_BACKWARD = struct.Struct("17q")


def lib() -> ctypes.CDLL:
    """The loaded library; raises if liblinear_norm.so has not been built."""
    global _lib, _dtypes
    if _lib is None:
        import torch
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
        _dtypes = {torch.float16: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2}
        _lib = L
    return _lib


class RMSNormResult(NamedTuple):
    y: object       # the normalised rows
    h: object       # x + residual (x itself without a residual)
    rstd: object    # float32, one a row; None unless asked for
    scale: object   # float32, one a row; None unless y is in 8 bits


def _code(t, what, allowed=(0, 1)):
    c = _dtypes.get(t.dtype)
    if c not in allowed:
        raise ValueError(f"{what} has dtype {t.dtype}; it must be float16 or bfloat16"
                         + (" or float8_e4m3fn" if 2 in allowed else ""))
    return c


def _check(t, what, shape, dtype, device):
    """A tensor of the given shape and type on the call's device, with a unit column stride."""
    if t.shape != shape:
        raise ValueError(f"{what} is {tuple(t.shape)}; the call needs {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{what} has dtype {t.dtype}; the call needs {dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}; the call is on {device}")
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what} must be contiguous along its last dimension")


def _on_gpu(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.device


class _Call:
    """Device and stream of one call: torch allocates on the stream that the kernels run on, so
    that memory freed on return is handed out again only to work behind them."""

    __slots__ = ("torch", "stream", "handle", "context")

    def __init__(self, device, stream):
        import torch
        self.torch = torch
        self.context = []
        if torch.cuda.current_device() != device.index:
            self.context.append(torch.cuda.device(device))
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
            self.context.append(torch.cuda.stream(stream))
        self.stream = stream

    def __enter__(self):
        for c in self.context:
            c.__enter__()
        s = self.torch.cuda.current_stream() if self.stream is None else self.stream
        self.handle = s.cuda_stream
        return self

    def __exit__(self, *exc):
        for c in reversed(self.context):
            c.__exit__(*exc)
        return False


def _run(name, device, packed, with_workspace):
    """Calls the library; `packed(ws, bytes)` gives the arguments.  A workspace is allocated
    only where the call asks for one."""
    import torch
    L = lib()
    f = getattr(L, name)
    rc = f(packed(0, 0))
    if rc == _pkg.ERR_WORKSPACE and with_workspace:
        need = getattr(L, name + "_workspace")(packed(0, 0))
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        rc = f(packed(ws.data_ptr(), need))
    if rc != _pkg.OK:
        raise _pkg.GemmError(rc, name)


def _row(t):
    """(pointer, row stride) of a matrix, or of nothing."""
    return (0, 0) if t is None else (t.data_ptr(), t.stride(0))


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def linear(a, b, bias=None, residual=None, *, activation="none", scale_a=None, scale_b=None,
           out_dtype=None, with_pre=False, out=None, stream=None):
    """act(a @ b + bias) + residual on the GPU: fp32 sums, one rounding.

    a (m, k) and b (k, n): float16 or bfloat16, each row- or column-major with any leading
    dimension (a weight stored (n, k) is passed as `w.t()`); or float8_e4m3fn, k-contiguous (a
    row-major, b column-major) with 16-byte aligned rows, and `scale_a` (m,) and `scale_b` (n,)
    float32 factors of the rows and columns (1 if not given).  bias (n,), residual (m, n): of
    the output's type, which is the operands' (8-bit operands: `out_dtype`, bfloat16 if not
    given).  activation: none, relu, gelu, gelu_tanh or silu.  Returns the (m, n) result, or
    (result, pre) with `with_pre`, where pre is the value before the activation, which
    linear_backward needs.  `out` may be the residual's own tensor.
    """
    import torch
    L = lib()
    device = _on_gpu(a, "a")
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("expected 2-D operands")
    m, k = a.shape
    n = b.shape[1]
    ty = _code(a, "a", (0, 1, 2))
    if b.shape[0] != k or b.dtype != a.dtype or b.device != device:
        raise ValueError(f"b is {tuple(b.shape)} of {b.dtype} on {b.device}; a is "
                         f"{tuple(a.shape)} of {a.dtype} on {device}")
    if ty == 2:
        out_dtype = out_dtype or torch.bfloat16
        if _dtypes.get(out_dtype) not in (0, 1):
            raise ValueError(f"out_dtype must be float16 or bfloat16, got {out_dtype}")
    elif out_dtype not in (None, a.dtype):
        raise ValueError(f"out_dtype is the operands' type, {a.dtype}; got {out_dtype}")
    else:
        out_dtype = a.dtype
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}; got {activation!r}")
    if bias is not None:
        _check(bias, "bias", (n,), out_dtype, device)
    if residual is not None:
        _check(residual, "residual", (m, n), out_dtype, device)
    if scale_a is not None:
        _check(scale_a, "scale_a", (m,), torch.float32, device)
    if scale_b is not None:
        _check(scale_b, "scale_b", (n,), torch.float32, device)
    if out is not None:
        _check(out, "out", (m, n), out_dtype, device)
    with _Call(device, stream) as call:
        if out is None:
            out = torch.empty((m, n), dtype=out_dtype, device=device)
        pre = torch.empty((m, n), dtype=out_dtype, device=device) if with_pre else None
        _run("linear_forward", device, lambda ws, nbytes: _FORWARD.pack(
            m, n, k, ty, _dtypes[out_dtype], ACTIVATIONS[activation],
            a.data_ptr(), *a.stride(), b.data_ptr(), *b.stride(), _ptr(scale_a), _ptr(scale_b),
            _ptr(bias), *_row(residual), *_row(out), *_row(pre), ws, nbytes, call.handle), True)
    return (out, pre) if with_pre else out


def linear_backward(dc, a, b, pre=None, *, activation="none", bias_grad=False, a_grad=True,
                    b_grad=True, stream=None):
    """(da, db, dbias): gradients of linear's a, b and bias (None where not asked for).

    dc (m, n) is the gradient of linear's result; that of its residual is dc itself.  pre (m, n)
    is linear's value before the activation (not needed for "none").  All of one 16-bit type;
    dc and pre contiguous along n, a and b as in linear.  db has b's storage order.
    """
    import torch
    lib()
    device = _on_gpu(dc, "dc")
    ty = _code(dc, "dc")
    if dc.dim() != 2 or a.dim() != 2 or b.dim() != 2:
        raise ValueError("expected 2-D operands")
    m, n = dc.shape
    k = a.shape[1]
    _check(dc, "dc", (m, n), dc.dtype, device)
    for t, what, shape in ((a, "a", (m, k)), (b, "b", (k, n))):
        if t.shape != shape or t.dtype != dc.dtype or t.device != device:
            raise ValueError(f"{what} is {tuple(t.shape)} of {t.dtype} on {t.device}; the call "
                             f"needs {shape} of {dc.dtype} on {device}")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}; got {activation!r}")
    if activation != "none":
        if pre is None:
            raise ValueError(f"the gradient of {activation} needs pre")
        _check(pre, "pre", (m, n), dc.dtype, device)
    with _Call(device, stream) as call:
        da = torch.empty((m, k), dtype=dc.dtype, device=device) if a_grad else None
        db = None
        if b_grad:
            columns = b.stride(0) == 1 and b.stride(1) != 1
            db = (torch.empty((n, k), dtype=dc.dtype, device=device).t() if columns else
                  torch.empty((k, n), dtype=dc.dtype, device=device))
        dbias = torch.empty((n,), dtype=dc.dtype, device=device) if bias_grad else None
        _run("linear_backward", device, lambda ws, nbytes: _BACKWARD.pack(
            m, n, k, ty, ACTIVATIONS[activation], *_row(dc), a.data_ptr(), *a.stride(),
            b.data_ptr(), *b.stride(), *_row(pre), *_row(da),
            *((0, 0, 0) if db is None else (db.data_ptr(), *db.stride())), _ptr(dbias),
            ws, nbytes, call.handle), True)
    return da, db, dbias


def _rows_aligned(torch, rows, dim, dtype, device):
    """rows x dim bytes whose rows start on 16-byte boundaries (what linear reads)."""
    pad = -(-dim // 16) * 16
    t = torch.empty((rows, pad), dtype=dtype, device=device)
    return t if pad == dim else t[:, :dim]


def rms_norm(x, weight, residual=None, *, eps=1e-5, out_dtype=None, with_rstd=False,
             stream=None):
    """RMSNormResult of h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.

    x, residual (rows, dim) and weight (dim,): one 16-bit type, rows contiguous, any row stride.
    y has that type, or with out_dtype=torch.float8_e4m3fn it is y / scale in 8 bits, with one
    float32 scale a row, laid out as linear's 8-bit operand.  h is rounded to x's type; the norm
    is taken of the unrounded sum.  `with_rstd` also returns 1 / sqrt(mean(h^2) + eps), which
    rms_norm_backward needs.
    """
    import torch
    lib()
    device = _on_gpu(x, "x")
    ty = _code(x, "x")
    if x.dim() != 2:
        raise ValueError("expected a 2-D x")
    rows, dim = x.shape
    _check(x, "x", (rows, dim), x.dtype, device)
    _check(weight, "weight", (dim,), x.dtype, device)
    if residual is not None:
        _check(residual, "residual", (rows, dim), x.dtype, device)
    out_dtype = out_dtype or x.dtype
    q8 = out_dtype == torch.float8_e4m3fn
    if not q8 and out_dtype != x.dtype:
        raise ValueError(f"out_dtype must be {x.dtype} or float8_e4m3fn, got {out_dtype}")
    with _Call(device, stream) as call:
        y = (_rows_aligned(torch, rows, dim, out_dtype, device) if q8 else
             torch.empty((rows, dim), dtype=out_dtype, device=device))
        h = None if residual is None else torch.empty((rows, dim), dtype=x.dtype, device=device)
        scale = torch.empty((rows,), dtype=torch.float32, device=device) if q8 else None
        rstd = torch.empty((rows,), dtype=torch.float32, device=device) if with_rstd else None
        _run("rms_norm_forward", device, lambda ws, nbytes: _NORM.pack(
            rows, dim, ty, _dtypes[out_dtype], *_row(x), *_row(residual), weight.data_ptr(),
            *_row(y), _ptr(scale), *_row(h), _ptr(rstd), float(eps), call.handle), False)
    return RMSNormResult(y, x if h is None else h, rstd, scale)


def rms_norm_backward(dy, h, weight, rstd, *, dh=None, weight_grad=True, stream=None):
    """(dx, dweight) of rms_norm: dx is the gradient of x and of the residual alike.

    dy (rows, dim): gradient of y; h and rstd as rms_norm returned them; dh: the gradient that
    reaches h by another way (the residual stream), added to dx.
    """
    import torch
    lib()
    device = _on_gpu(dy, "dy")
    ty = _code(dy, "dy")
    if dy.dim() != 2:
        raise ValueError("expected a 2-D dy")
    rows, dim = dy.shape
    _check(dy, "dy", (rows, dim), dy.dtype, device)
    _check(h, "h", (rows, dim), dy.dtype, device)
    _check(weight, "weight", (dim,), dy.dtype, device)
    _check(rstd, "rstd", (rows,), torch.float32, device)
    if dh is not None:
        _check(dh, "dh", (rows, dim), dy.dtype, device)
    with _Call(device, stream) as call:
        dx = torch.empty((rows, dim), dtype=dy.dtype, device=device)
        dweight = torch.empty((dim,), dtype=dy.dtype, device=device) if weight_grad else None
        _run("rms_norm_backward", device, lambda ws, nbytes: _NORM_BACKWARD.pack(
            rows, dim, ty, *_row(dy), *_row(h), weight.data_ptr(), rstd.data_ptr(), *_row(dh),
            *_row(dx), _ptr(dweight), ws, nbytes, call.handle), True)
    return dx, dweight
