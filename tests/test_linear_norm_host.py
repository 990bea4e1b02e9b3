"""The linear layer's and the norm's argument checks, workspace sizes and Python checks, on the
CPU: every call here is refused, or has nothing to launch, so pointers are only numbers."""
import ctypes
import os
import struct

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from dense_gemm_f16f32_amd import linear_norm as ln  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(ln.LIB_PATH), reason="library not built")

F16, BF16, E4M3 = 0, 1, 2
FORWARD = ("m n k type out_type activation a a_row a_col b b_row b_col scale_a scale_b bias "
           "residual residual_row out out_row pre pre_row workspace workspace_bytes stream").split()
BACKWARD = ("m n k type activation dc dc_row a a_row a_col b b_row b_col pre pre_row da da_row "
            "db db_row db_col dbias workspace workspace_bytes stream").split()
NORM = ("rows dim type out_type x x_row residual residual_row weight y y_row scale h h_row rstd "
        "eps stream").split()
NORM_BACKWARD = ("rows dim type dy dy_row h h_row weight rstd dh dh_row dx dx_row dweight "
                 "workspace workspace_bytes stream").split()
# the argument structures are arrays of 8-byte fields
FORWARD_STRUCT = BACKWARD_STRUCT = struct.Struct("24q")
NORM_STRUCT = struct.Struct("15qdq")
NORM_BACKWARD_STRUCT = struct.Struct("17q")
G = 1 << 44   # spacing of the made-up addresses


def args(names, layout, base, **change):
    d = dict.fromkeys(names, 0)
    d.update(base)
    d.update(change)
    assert set(d) == set(names)
    return layout.pack(*(d[n] for n in names))


def forward(call="linear_forward", **change):
    base = dict(m=64, n=96, k=128, type=F16, out_type=F16, a=G, a_row=128, a_col=1, b=2 * G,
                b_row=96, b_col=1, bias=3 * G, residual=4 * G, residual_row=96, out=5 * G,
                out_row=96, pre=6 * G, pre_row=96)
    return getattr(ln.lib(), call)(args(FORWARD, FORWARD_STRUCT, base, **change))


def forward8(**change):
    base = dict(type=E4M3, a_row=128, b_row=1, b_col=128, scale_a=7 * G, scale_b=8 * G)
    return forward(**{**base, **change})


def backward(call="linear_backward", **change):
    base = dict(m=64, n=96, k=128, type=BF16, activation=4, dc=G, dc_row=96, a=2 * G, a_row=128,
                a_col=1, b=3 * G, b_row=1, b_col=128, pre=4 * G, pre_row=96, da=5 * G, da_row=128,
                db=6 * G, db_row=1, db_col=128, dbias=7 * G, workspace=8 * G,
                workspace_bytes=G)
    return getattr(ln.lib(), call)(args(BACKWARD, BACKWARD_STRUCT, base, **change))


def norm(**change):
    base = dict(rows=4, dim=64, type=F16, out_type=F16, x=G, x_row=64, residual=2 * G,
                residual_row=64, weight=3 * G, y=4 * G, y_row=64, h=5 * G, h_row=64, rstd=6 * G,
                eps=1e-5)
    return ln.lib().rms_norm_forward(args(NORM, NORM_STRUCT, base, **change))


def norm_backward(call="rms_norm_backward", **change):
    base = dict(rows=400, dim=64, type=F16, dy=G, dy_row=64, h=2 * G, h_row=64, weight=3 * G,
                rstd=4 * G, dh=5 * G, dh_row=64, dx=6 * G, dx_row=64, dweight=7 * G,
                workspace=8 * G, workspace_bytes=G)
    return getattr(ln.lib(), call)(args(NORM_BACKWARD, NORM_BACKWARD_STRUCT, base, **change))


def test_null_arguments():
    for name in ("linear_forward", "linear_backward", "rms_norm_forward", "rms_norm_backward",
                 "linear_forward_workspace", "linear_backward_workspace",
                 "rms_norm_backward_workspace"):
        assert getattr(ln.lib(), name)(None) == g.ERR_NULL


@pytest.mark.parametrize("change,code", [
    (dict(m=-1), g.ERR_DIM), (dict(n=1 << 31), g.ERR_DIM), (dict(k=-5), g.ERR_DIM),
    (dict(type=3), g.ERR_OPTS), (dict(type=-1), g.ERR_OPTS), (dict(out_type=BF16), g.ERR_OPTS),
    (dict(out_type=E4M3), g.ERR_OPTS), (dict(activation=5), g.ERR_OPTS),
    (dict(activation=-1), g.ERR_OPTS), (dict(scale_a=7 * G), g.ERR_OPTS),
    (dict(a=0), g.ERR_NULL), (dict(b=0), g.ERR_NULL), (dict(out=0), g.ERR_NULL),
    (dict(a=G + 1), g.ERR_OPTS), (dict(out=5 * G + 1), g.ERR_OPTS), (dict(bias=3 * G + 1), g.ERR_OPTS),
    (dict(a_row=127), g.ERR_LD), (dict(a_row=128, a_col=2), g.ERR_LD), (dict(b_row=95), g.ERR_LD),
    (dict(b_row=2, b_col=2), g.ERR_LD), (dict(out_row=95), g.ERR_LD), (dict(pre_row=-1), g.ERR_LD),
    (dict(residual_row=0), g.ERR_LD), (dict(out=G + 64), g.ERR_OVERLAP),
    (dict(out=3 * G), g.ERR_OVERLAP), (dict(pre=5 * G + 100), g.ERR_OVERLAP),
    (dict(out=4 * G + 2), g.ERR_OVERLAP), (dict(out=4 * G, out_row=128), g.ERR_OVERLAP),
    (dict(pre=4 * G), g.ERR_OVERLAP), (dict(a_row=1 << 60), g.ERR_TOO_LARGE),
    (dict(a_row=1 << 30), g.ERR_TOO_LARGE), (dict(b_row=1 << 30), g.ERR_TOO_LARGE)])
def test_forward_refusals(change, code):
    assert forward(**change) == code
    assert forward("linear_forward_workspace", **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(a=G + 8), g.ERR_OPTS), (dict(a_row=136), g.ERR_LD), (dict(b_col=136), g.ERR_LD),
    (dict(a_row=1, a_col=64), g.ERR_LD), (dict(b_row=96, b_col=1), g.ERR_LD),
    (dict(out_type=E4M3), g.ERR_OPTS), (dict(scale_a=7 * G + 2), g.ERR_OPTS),
    (dict(out=7 * G), g.ERR_OVERLAP), (dict(pre=8 * G), g.ERR_OVERLAP)])
def test_8_bit_refusals(change, code):
    assert forward8(**change) == code


def test_empty_results_need_nothing():
    nothing = dict.fromkeys(("a", "b", "bias", "residual", "out", "pre"), 0)
    for d in (dict(m=0), dict(n=0), dict(m=0, n=0, k=0)):
        assert forward(**d, **nothing) == g.OK
        assert forward("linear_forward_workspace", **d, **nothing) == 0


def test_split_k_workspace():
    """A deep product with few results asks for room for its k slices."""
    deep = dict(m=40, n=70, k=8192, a_row=8192, b_row=70, residual_row=70, out_row=70, pre_row=70)
    need = forward("linear_forward_workspace", **deep)
    assert need > 0
    assert forward(**deep) == g.ERR_WORKSPACE
    assert forward(**deep, workspace=9 * G, workspace_bytes=need - 1) == g.ERR_WORKSPACE
    assert forward(**deep, workspace=9 * G + 8, workspace_bytes=need) == g.ERR_WORKSPACE
    assert forward(**deep, workspace=2 * G, workspace_bytes=need) == g.ERR_OVERLAP


@pytest.mark.parametrize("change,code", [
    (dict(m=-1), g.ERR_DIM), (dict(type=E4M3), g.ERR_OPTS), (dict(activation=7), g.ERR_OPTS),
    (dict(dc=0), g.ERR_NULL), (dict(pre=0), g.ERR_NULL), (dict(a=0), g.ERR_NULL),
    (dict(b=0), g.ERR_NULL), (dict(dc_row=95), g.ERR_LD), (dict(da_row=127), g.ERR_LD),
    (dict(a_row=2, a_col=2), g.ERR_LD), (dict(db_row=2, db_col=2), g.ERR_LD),
    (dict(db_row=1, db_col=127), g.ERR_LD), (dict(dbias=7 * G + 1), g.ERR_OPTS),
    (dict(da=G), g.ERR_OVERLAP), (dict(db=3 * G), g.ERR_OVERLAP), (dict(dbias=4 * G), g.ERR_OVERLAP),
    (dict(da=6 * G + 64), g.ERR_OVERLAP)])
def test_backward_refusals(change, code):
    assert backward(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(workspace=0), g.ERR_WORKSPACE), (dict(workspace_bytes=100), g.ERR_WORKSPACE),
    (dict(workspace=8 * G + 4), g.ERR_WORKSPACE), (dict(workspace=2 * G), g.ERR_OVERLAP)])
def test_backward_workspace_refusals(change, code):
    """A large pass keeps dpre and partial sums in its workspace."""
    large = dict(m=4096, n=4096, k=4096, dc_row=4096, a_row=4096, b_col=4096, pre_row=4096,
                 da_row=4096, db_col=4096)
    assert backward("linear_backward_workspace", **large) >= 4096 * 4096 * 2
    assert backward(**large, **change) == code


def test_backward_with_nothing_to_do():
    none = dict(da=0, db=0, dbias=0)
    assert backward(**none, activation=0, workspace=0) == g.OK
    assert backward(m=0, n=0, k=0, workspace=0) == g.OK
    assert backward("linear_backward_workspace", **none, activation=0) == 0


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), g.ERR_DIM), (dict(dim=0), g.ERR_DIM), (dict(dim=1 << 31), g.ERR_DIM),
    (dict(type=E4M3), g.ERR_OPTS), (dict(out_type=BF16), g.ERR_OPTS), (dict(eps=-1.0), g.ERR_OPTS),
    (dict(eps=float("nan")), g.ERR_OPTS), (dict(scale=7 * G), g.ERR_OPTS),
    (dict(out_type=E4M3), g.ERR_NULL), (dict(x=0), g.ERR_NULL), (dict(weight=0), g.ERR_NULL),
    (dict(y=0), g.ERR_NULL), (dict(h=0), g.ERR_NULL), (dict(x_row=63), g.ERR_LD),
    (dict(y_row=0), g.ERR_LD), (dict(h_row=63), g.ERR_LD), (dict(x=G + 1), g.ERR_OPTS),
    (dict(rstd=6 * G + 2), g.ERR_OPTS), (dict(y=G), g.ERR_OVERLAP), (dict(y=3 * G), g.ERR_OVERLAP),
    (dict(h=G + 2), g.ERR_OVERLAP), (dict(h=2 * G, h_row=128), g.ERR_OVERLAP),
    (dict(rstd=4 * G), g.ERR_OVERLAP)])
def test_norm_refusals(change, code):
    assert norm(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), g.ERR_DIM), (dict(dim=0), g.ERR_DIM), (dict(type=E4M3), g.ERR_OPTS),
    (dict(dy=0), g.ERR_NULL), (dict(h=0), g.ERR_NULL), (dict(weight=0), g.ERR_NULL),
    (dict(rstd=0), g.ERR_NULL), (dict(dx=0), g.ERR_NULL), (dict(dy_row=63), g.ERR_LD),
    (dict(dx_row=63), g.ERR_LD), (dict(dweight=7 * G + 1), g.ERR_OPTS),
    (dict(workspace=0), g.ERR_WORKSPACE), (dict(workspace_bytes=16), g.ERR_WORKSPACE),
    (dict(dx=2 * G), g.ERR_OVERLAP), (dict(dx=G + 2), g.ERR_OVERLAP),
    (dict(dweight=6 * G), g.ERR_OVERLAP), (dict(workspace=2 * G), g.ERR_OVERLAP)])
def test_norm_backward_refusals(change, code):
    assert norm_backward(**change) == code


def test_norm_without_rows():
    assert norm(rows=0, x=0, residual=0, weight=0, y=0, h=0, rstd=0) == g.OK
    assert norm_backward("rms_norm_backward_workspace", rows=0) == 0
    assert norm_backward("rms_norm_backward_workspace", dweight=0) == 0
    # few rows: one workgroup, which needs none
    assert norm_backward("rms_norm_backward_workspace") > 0
    assert norm_backward("rms_norm_backward_workspace", rows=4) == 0


def test_structures_match_the_header():
    """Field names and count of the packed arguments against include/linear_norm.h."""
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "linear_norm.h")).read()
    for name, fields, layout in (("linear_forward_args", FORWARD, FORWARD_STRUCT),
                                 ("linear_backward_args", BACKWARD, BACKWARD_STRUCT),
                                 ("rms_norm_forward_args", NORM, NORM_STRUCT),
                                 ("rms_norm_backward_args", NORM_BACKWARD, NORM_BACKWARD_STRUCT)):
        body = re.search(r"typedef struct " + name + r" \{(.*?)\} ", text, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        found = [re.sub(r".*[ *]", "", f.strip()) for line in body.split(";") if line.strip()
                 for f in line.split(",")]
        assert found == fields and layout.size == 8 * len(fields)
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_python_checks():
    x = torch.zeros((4, 8), dtype=torch.float16)
    for call in (lambda: g.linear(x, x.t()), lambda: g.rms_norm(x, x[0]),
                 lambda: g.linear_backward(x, x, x),
                 lambda: g.rms_norm_backward(x, x, x[0], x[:, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
