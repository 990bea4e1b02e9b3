"""The layer norm's, the 8-bit rows' and the checkpoints' argument checks and workspace sizes, on the
CPU: every call here is refused, or has nothing to launch, so pointers are only numbers."""
import os
import re
import struct

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from dense_gemm_f16f32_amd import linear_norm as ln  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(ln.LIB_PATH), reason="library not built")

F16, BF16, E4M3, I8 = 0, 1, 2, 8
G = 1 << 44   # spacing of the made-up addresses
FORWARD = ("m n k type out_type activation a a_row a_col b b_row b_col scale_a scale_b bias "
           "residual residual_row out out_row pre pre_row workspace workspace_bytes stream").split()
BACKWARD = ("m n k type activation dc dc_row a a_row a_col b b_row b_col pre pre_row da da_row "
            "db db_row db_col dbias workspace workspace_bytes stream").split()
PACKED = "values values_row scale scale_row".split()
KEPT = "a a_activation pre".split()
NORM = ("rows dim type out_type x x_row residual residual_row weight bias y y_row scale h h_row mean "
        "rstd eps stream").split()
NORM_BACKWARD = ("rows dim type dy dy_row h h_row weight mean rstd dh dh_row dx dx_row dweight "
                 "dbias workspace workspace_bytes stream").split()
QUANTIZE = "rows dim type out_type x x_row values values_row scale stream".split()
PACK = "rows dim type x x_row out stream".split()
UNPACK = "rows dim type activation in y y_row stream".split()


def fields(names, base, change, eps=None):
    d = dict.fromkeys(names, 0)
    d.update(base)
    d.update(change)
    assert set(d) == set(names), set(d) ^ set(names)
    return struct.pack("".join("d" if n == eps else "q" for n in names), *(d[n] for n in names))


def packed(at, cols, **change):
    return fields(PACKED, dict(values=at, values_row=cols, scale=at + G // 2,
                               scale_row=-(-cols // 32)), change)


def norm(call="layer_norm_forward", **change):
    base = dict(rows=4, dim=64, type=F16, out_type=F16, x=G, x_row=64, residual=2 * G,
                residual_row=64, weight=3 * G, bias=7 * G, y=4 * G, y_row=64, h=5 * G, h_row=64,
                mean=8 * G, rstd=6 * G, eps=1e-5)
    return getattr(ln.lib(), call)(fields(NORM, base, change, "eps"))


def norm_backward(call="layer_norm_backward", **change):
    base = dict(rows=4000, dim=64, type=F16, dy=G, dy_row=64, h=2 * G, h_row=64, weight=3 * G,
                mean=4 * G, rstd=5 * G, dh=6 * G, dh_row=64, dx=7 * G, dx_row=64, dweight=8 * G,
                dbias=9 * G, workspace=10 * G, workspace_bytes=G)
    return getattr(ln.lib(), call)(fields(NORM_BACKWARD, base, change))


def quantize(**change):
    base = dict(rows=4, dim=64, type=BF16, out_type=I8, x=G, x_row=64, values=2 * G, values_row=64,
                scale=3 * G)
    return ln.lib().quantize_rows(fields(QUANTIZE, base, change))


def pack(out=None, **change):
    base = dict(rows=4, dim=70, type=BF16, x=G, x_row=70)
    d = {**dict.fromkeys(PACK, 0), **base, **change}
    head = struct.pack("5q", *(d[n] for n in PACK[:5]))
    return ln.lib().pack8(head + (out or packed(2 * G, 70)) + struct.pack("q", 0))


def unpack(src=None, **change):
    d = {**dict(rows=4, dim=70, type=BF16, activation=0, y=G, y_row=70), **change}
    head = struct.pack("4q", *(d[n] for n in UNPACK[:4]))
    return ln.lib().unpack8(head + (src or packed(2 * G, 70))
                            + struct.pack("3q", d["y"], d["y_row"], 0))


def forward(pre, call="linear_forward_packed", **change):
    base = dict(m=64, n=96, k=128, type=F16, out_type=F16, a=G, a_row=128, a_col=1, b=2 * G,
                b_row=96, b_col=1, bias=3 * G, residual=4 * G, residual_row=96, out=5 * G,
                out_row=96)
    return getattr(ln.lib(), call)(fields(FORWARD, base, change), pre)


def backward(a=None, pre=None, a_activation=0, call="linear_backward_packed", **change):
    """a, pre: packed, or None for the ones in 16 bits."""
    base = dict(m=64, n=96, k=128, type=BF16, activation=4, dc=G, dc_row=96,
                a=0 if a else 2 * G, a_row=128, a_col=1, b=3 * G, b_row=1, b_col=128,
                pre=0 if pre else 4 * G, pre_row=96, da=5 * G, da_row=128, db=6 * G, db_row=1,
                db_col=128, dbias=7 * G, workspace=8 * G, workspace_bytes=G)
    none = bytes(8 * len(PACKED))
    kept = (a or none) + struct.pack("q", a_activation) + (pre or none)
    return getattr(ln.lib(), call)(fields(BACKWARD, base, change), kept)


def test_structures_match_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "linear_norm.h")) as f:
        text = f.read()
    for name, want in (("layer_norm_forward_args", NORM),
                       ("layer_norm_backward_args", NORM_BACKWARD),
                       ("quantize_rows_args", QUANTIZE), ("packed8_matrix", PACKED),
                       ("pack8_args", PACK), ("unpack8_args", UNPACK), ("linear_kept", KEPT)):
        body = re.search(r"typedef struct " + name + r" \{(.*?)\} ", text, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        found = [re.sub(r".*[ *]", "", x.strip()) for line in body.split(";") if line.strip()
                 for x in line.split(",")]
        assert found == want


def test_null_arguments():
    L = ln.lib()
    for name in ("layer_norm_forward", "layer_norm_backward", "layer_norm_backward_workspace",
                 "quantize_rows", "pack8", "unpack8"):
        assert getattr(L, name)(None) == g.ERR_NULL
    for name in ("linear_forward_packed", "linear_backward_packed",
                 "linear_forward_packed_workspace", "linear_backward_packed_workspace"):
        assert getattr(L, name)(None, None) == g.ERR_NULL


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), g.ERR_DIM), (dict(dim=0), g.ERR_DIM), (dict(dim=1 << 31), g.ERR_DIM),
    (dict(type=E4M3), g.ERR_OPTS), (dict(type=I8), g.ERR_OPTS), (dict(type=3), g.ERR_OPTS),
    (dict(out_type=BF16), g.ERR_OPTS), (dict(out_type=3), g.ERR_OPTS),
    (dict(eps=-1.0), g.ERR_OPTS), (dict(eps=float("nan")), g.ERR_OPTS),
    (dict(scale=9 * G), g.ERR_OPTS), (dict(out_type=I8), g.ERR_NULL), (dict(x=0), g.ERR_NULL),
    (dict(y=0), g.ERR_NULL), (dict(h=0), g.ERR_NULL), (dict(weight=0), g.ERR_NULL),
    (dict(x_row=63), g.ERR_LD), (dict(h_row=63), g.ERR_LD), (dict(x=G + 1), g.ERR_OPTS),
    (dict(bias=7 * G + 1), g.ERR_OPTS), (dict(mean=8 * G + 2), g.ERR_OPTS),
    (dict(rstd=6 * G + 2), g.ERR_OPTS), (dict(x_row=1 << 60), g.ERR_TOO_LARGE),
    (dict(y=G), g.ERR_OVERLAP), (dict(y=7 * G), g.ERR_OVERLAP), (dict(mean=6 * G), g.ERR_OVERLAP),
    (dict(mean=4 * G), g.ERR_OVERLAP), (dict(h=7 * G), g.ERR_OVERLAP),
    (dict(h=G + 2), g.ERR_OVERLAP), (dict(h=G, h_row=65), g.ERR_OVERLAP)])
def test_layer_norm_refusals(change, code):
    assert norm(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=1 << 31), g.ERR_DIM), (dict(dim=0), g.ERR_DIM), (dict(type=I8), g.ERR_OPTS),
    (dict(dy=0), g.ERR_NULL), (dict(h=0), g.ERR_NULL), (dict(dx=0), g.ERR_NULL),
    (dict(weight=0), g.ERR_NULL), (dict(mean=0), g.ERR_NULL), (dict(rstd=0), g.ERR_NULL),
    (dict(dh_row=63), g.ERR_LD), (dict(dbias=9 * G + 1), g.ERR_OPTS),
    (dict(mean=4 * G + 2), g.ERR_OPTS), (dict(workspace=0), g.ERR_WORKSPACE),
    (dict(workspace_bytes=100), g.ERR_WORKSPACE), (dict(workspace=10 * G + 8), g.ERR_WORKSPACE),
    (dict(dbias=8 * G), g.ERR_OVERLAP), (dict(dbias=10 * G), g.ERR_OVERLAP),
    (dict(dx=2 * G), g.ERR_OVERLAP), (dict(dx=4 * G), g.ERR_OVERLAP),
    (dict(dx=G + 2), g.ERR_OVERLAP), (dict(dbias=G), g.ERR_OVERLAP)])
def test_layer_norm_backward_refusals(change, code):
    assert norm_backward(**change) == code


def test_layer_norm_workspace():
    size = lambda **c: norm_backward("layer_norm_backward_workspace", **c)  # noqa: E731
    both = size()
    assert both > 0 and size(dweight=0) == size(dbias=0) == both // 2
    assert size(dweight=0, dbias=0) == 0 and size(rows=1024) == size(rows=4) == 0 and size(dim=0) == g.ERR_DIM


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), g.ERR_DIM), (dict(dim=0), g.ERR_DIM), (dict(type=I8), g.ERR_OPTS),
    (dict(out_type=BF16), g.ERR_OPTS), (dict(x=0), g.ERR_NULL), (dict(values=0), g.ERR_NULL),
    (dict(scale=0), g.ERR_NULL), (dict(scale=3 * G + 2), g.ERR_OPTS), (dict(x_row=63), g.ERR_LD),
    (dict(values_row=63), g.ERR_LD), (dict(values=G), g.ERR_OVERLAP),
    (dict(scale=2 * G), g.ERR_OVERLAP)])
def test_quantize_refusals(change, code):
    assert quantize(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), g.ERR_DIM), (dict(dim=1 << 31), g.ERR_DIM), (dict(type=E4M3), g.ERR_OPTS),
    (dict(x=0), g.ERR_NULL), (dict(x_row=69), g.ERR_LD), (dict(x=G + 1), g.ERR_OPTS),
    (dict(out=packed(0, 70)), g.ERR_NULL), (dict(out=packed(2 * G, 70, scale=0)), g.ERR_NULL),
    (dict(out=packed(2 * G, 69)), g.ERR_LD), (dict(out=packed(2 * G, 70, scale_row=2)), g.ERR_LD),
    (dict(out=packed(G, 70)), g.ERR_OVERLAP),
    (dict(out=packed(2 * G, 70, scale=2 * G + 279)), g.ERR_OVERLAP)])
def test_pack_refusals(change, code):
    assert pack(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), g.ERR_DIM), (dict(type=I8), g.ERR_OPTS), (dict(activation=5), g.ERR_OPTS),
    (dict(activation=-1), g.ERR_OPTS), (dict(y=0), g.ERR_NULL), (dict(y_row=69), g.ERR_LD),
    (dict(y=G + 1), g.ERR_OPTS), (dict(src=packed(0, 70)), g.ERR_NULL),
    (dict(src=packed(2 * G, 70, scale_row=2)), g.ERR_LD), (dict(y=2 * G), g.ERR_OVERLAP)])
def test_unpack_refusals(change, code):
    assert unpack(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(pre=packed(0, 96)), g.ERR_NULL), (dict(pre=packed(6 * G, 95)), g.ERR_LD),
    (dict(pre=packed(6 * G, 96, scale_row=2)), g.ERR_LD),
    (dict(pre=packed(5 * G, 96)), g.ERR_OVERLAP), (dict(pre=packed(G, 96)), g.ERR_OVERLAP),
    (dict(pre=packed(4 * G, 96)), g.ERR_OVERLAP),
    (dict(pre=packed(6 * G, 96, scale=4 * G)), g.ERR_OVERLAP),
    (dict(pre=packed(6 * G, 96, scale=6 * G)), g.ERR_OVERLAP),
    (dict(pre=packed(6 * G, 96), type=3), g.ERR_OPTS)])
def test_forward_refusals(change, code):
    assert forward(**change) == code


def test_forward_takes_one_form_of_pre():
    args = dict(m=64, n=96, k=128, type=F16, out_type=F16, a=G, a_row=128, a_col=1, b=2 * G,
                b_row=96, b_col=1, out=5 * G, out_row=96, pre=7 * G, pre_row=96)
    assert ln.lib().linear_forward_packed(fields(FORWARD, args, {}), packed(6 * G, 96)) == g.ERR_OPTS


def test_int8_operands():
    """Their bounds are e4m3's, and k stays below 2^17."""
    base = dict(type=I8, a_row=128, b_row=1, b_col=128, scale_a=7 * G, scale_b=8 * G)
    for change, code in ((dict(k=1 << 17, a_row=1 << 17, b_col=1 << 17), g.ERR_TOO_LARGE),
                         (dict(a=G + 8), g.ERR_OPTS), (dict(a_row=136), g.ERR_LD),
                         (dict(b_row=96, b_col=1), g.ERR_LD), (dict(out_type=I8), g.ERR_OPTS),
                         (dict(scale_a=7 * G + 2), g.ERR_OPTS), (dict(out=7 * G), g.ERR_OVERLAP)):
        assert forward(None, **{**base, **change}) == code
    assert forward(None, call="linear_forward_packed_workspace", **base) == 0
    deep = dict(base, m=1, n=32, k=131071, a_row=131072, b_col=131072)
    assert forward(None, call="linear_forward_packed_workspace", **deep) > 0


@pytest.mark.parametrize("change,code", [
    (dict(a=packed(2 * G, 127)), g.ERR_LD), (dict(a=packed(2 * G, 128, scale=0)), g.ERR_NULL),
    (dict(pre=packed(4 * G, 95)), g.ERR_LD), (dict(pre=packed(4 * G, 96, scale_row=1)), g.ERR_LD),
    (dict(a_activation=4), g.ERR_OPTS), (dict(a=packed(2 * G, 128), a_activation=5), g.ERR_OPTS),
    (dict(a=packed(5 * G, 128)), g.ERR_OVERLAP), (dict(pre=packed(7 * G, 96)), g.ERR_OVERLAP),
    (dict(a=packed(8 * G, 128)), g.ERR_OVERLAP),
    (dict(a=packed(2 * G, 128), workspace_bytes=64 * 128 * 2), g.ERR_WORKSPACE)])
def test_backward_refusals(change, code):
    assert backward(**change) == code


def test_backward_takes_one_form_of_each():
    kept = packed(2 * G, 128) + struct.pack("q", 0) + bytes(32)
    args = dict(m=64, n=96, k=128, type=BF16, dc=G, dc_row=96, a=9 * G, a_row=128, a_col=1,
                b=3 * G, b_row=1, b_col=128, db=6 * G, db_row=1, db_col=128)
    assert ln.lib().linear_backward_packed(fields(BACKWARD, args, {}), kept) == g.ERR_OPTS


def test_backward_workspace():
    def size(**c):
        return backward(call="linear_backward_packed_workspace", dc_row=960, pre_row=960, **c)

    plain = size(m=640, n=960)
    assert plain > 0
    # a restored in 16 bits, rows of whole 128 bytes
    assert size(a=packed(2 * G, 128), m=640, n=960) == plain + 640 * 128 * 2
    assert size(pre=packed(4 * G, 960), m=640, n=960) == plain
    assert size(a=packed(2 * G, 128), m=640, n=960, db=0) < plain + 640 * 128 * 2


def test_nothing_to_do():
    for call in (lambda: norm(rows=0), lambda: quantize(rows=0), lambda: pack(rows=0),
                 lambda: pack(dim=0), lambda: unpack(rows=0),
                 lambda: forward(packed(0, 0), m=0), lambda: forward(packed(0, 0), n=0),
                 lambda: norm_backward(rows=0, dweight=0, dbias=0)):
        assert call() == g.OK


def test_python_checks():
    x = torch.zeros((4, 8), dtype=torch.float16)
    p = g.Packed8(torch.zeros((4, 8), dtype=torch.int8),
                  torch.zeros((4, 1)).to(torch.float8_e8m0fnu))
    for call in (lambda: g.layer_norm(x, x[0]), lambda: g.quantize_rows(x), lambda: g.pack8(x),
                 lambda: g.layer_norm_backward(x, x, x[0], x[:, 0], x[:, 0]),
                 lambda: g.unpack8(p), lambda: g.linear_backward(x, p, x, p)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: g.layer_norm(None, x[0]), lambda: g.layer_norm(x, None),
                 lambda: g.quantize_rows(None), lambda: g.pack8(3), lambda: g.unpack8(x),
                 lambda: g.unpack8((p.values, p.scale)),
                 lambda: g.layer_norm_backward(x, x, x[0], None, x[:, 0])):
        with pytest.raises(TypeError):
            call()
