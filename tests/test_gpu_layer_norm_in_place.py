"""Layer norm results in their inputs' own memory, which the C functions allow and the Python functions
never ask for: h in x's or the residual's, dx in dy's or dh's.  Equal to the results in memory of
their own (the weight's and bias' gradients to their rounding: in place they are summed in another
order), for every row shape, for few rows and many, and for rows of any alignment."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from dense_gemm_f16f32_amd import linear_norm as ln  # noqa: E402
from linear_norm_util import F32, assert_close, normal, strided  # noqa: E402
from test_packed_host import NORM, NORM_BACKWARD, fields  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, E4M3, I8 = 1, 2, 8
DIMS = [3, 8, 100, 512, 1021, 1024, 2048, 4093, 4096, 8191, 16384, 20001]


def call(name, names, tensors, floating=None, **values):
    """A C entry point on tensors (given by field name, with their row strides)."""
    for field, t in tensors.items():
        values[field] = t.data_ptr()
        if field + "_row" in names:
            values[field + "_row"] = t.stride(0)
    values["stream"] = torch.cuda.current_stream().cuda_stream
    assert getattr(ln.lib(), name)(fields(names, {}, values, floating)) == g.OK


def inputs(dim, rows):
    q = torch.Generator(device="cuda")
    q.manual_seed(dim)
    pad = dim % 3
    return (lambda: strided(normal(q, (rows, dim), torch.bfloat16), pad, pad % 2),
            normal(q, (dim,), torch.bfloat16, 0.2) + 1, normal(q, (dim,), torch.bfloat16))


def like(t):
    """A tensor of t's strides, NaN around it, with t's values."""
    return strided(t, t.stride(0) - t.shape[1], t.storage_offset())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dim", DIMS)
def test_h_in_an_inputs_memory(dim, out):
    rows = 37
    make, w, b = inputs(dim, rows)
    x, res = make(), make()
    want = g.layer_norm(x, w, b, res, with_stats=True, out_dtype=out)
    for where in ("x", "residual"):
        t = {"x": like(x), "residual": like(res), "weight": w, "bias": b,
             "y": torch.empty((rows, -(-dim // 16) * 16), dtype=out, device="cuda")[:, :dim],
             "mean": torch.empty(rows, device="cuda"), "rstd": torch.empty(rows, device="cuda")}
        t["h"] = t[where]
        if want.scale is not None:
            t["scale"] = torch.empty(rows, device="cuda")
        call("layer_norm_forward", NORM, t, "eps", rows=rows, dim=dim, type=BF16, eps=1e-5,
             out_type={torch.bfloat16: BF16, torch.int8: I8}.get(out, E4M3))
        assert torch.equal(t["h"], want.h) and torch.equal(t["rstd"], want.rstd)
        assert torch.equal(t["mean"], want.mean) and torch.equal(t["y"].float(), want.y.float())
        other = "residual" if where == "x" else "x"
        assert torch.equal(t[other], {"x": x, "residual": res}[other])
        if want.scale is not None:
            assert torch.equal(t["scale"], want.scale)


@pytest.mark.parametrize("rows", [1, 700, 1500])
@pytest.mark.parametrize("dim", DIMS)
def test_dx_in_an_inputs_memory(dim, rows):
    make, w, _ = inputs(dim, rows)
    dy, dh, h = make(), make(), make()
    mean, rstd = torch.rand(rows, device="cuda") - 0.5, torch.rand(rows, device="cuda") + 0.5
    dx, dw, db = g.layer_norm_backward(dy, h, w, mean, rstd, dh=dh)
    d64 = dy.double()
    t64 = d64 * (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for where in ("dy", "dh"):
        t = {"dy": like(dy), "dh": like(dh), "h": h, "weight": w, "mean": mean, "rstd": rstd,
             "dweight": torch.empty(dim, dtype=w.dtype, device="cuda"),
             "dbias": torch.empty(dim, dtype=w.dtype, device="cuda")}
        t["dx"] = t[where]
        ws = torch.empty((2 * 1024 * (dim + 32),), device="cuda")
        t["workspace"] = ws
        call("layer_norm_backward", NORM_BACKWARD, t, rows=rows, dim=dim, type=BF16,
             workspace_bytes=ws.numel() * 4)
        assert torch.equal(t["dx"], dx)
        # a difference and a product rounded once each, the sum (rows + 16) 2^-23 of the magnitudes
        assert_close(t["dweight"], t64.sum(0), (rows + 20) * F32 * t64.abs().sum(0))
        assert_close(t["dbias"], d64.sum(0), (rows + 16) * F32 * d64.abs().sum(0))
        if where == "dh":
            assert torch.equal(t["dweight"], dw) and torch.equal(t["dbias"], db)
