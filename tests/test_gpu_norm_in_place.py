"""Results in their inputs' own memory, which the C functions allow and the Python functions never
ask for: h in x's or the residual's, dx in dy's or dh's.  Equal to the results in memory of their
own, for every row shape and for rows of any alignment."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from dense_gemm_f16f32_amd import linear_norm as ln  # noqa: E402
from linear_norm_util import normal, strided  # noqa: E402
from test_linear_norm_host import (NORM, NORM_BACKWARD, NORM_BACKWARD_STRUCT,  # noqa: E402
                                   NORM_STRUCT, args)

pytestmark = pytest.mark.gpu

BF16, E4M3 = 1, 2
# row shapes of one to sixteen waves and rows that no registers hold; odd row ends
DIMS = [3, 8, 100, 512, 1021, 1024, 2048, 4093, 4096, 8191, 16384, 20001]


def call(name, names, layout, tensors, **values):
    """A C entry point on tensors (given by field name, with their row strides)."""
    fields = dict(values, stream=torch.cuda.current_stream().cuda_stream)
    for field, t in tensors.items():
        fields[field] = t.data_ptr()
        if field + "_row" in names:
            fields[field + "_row"] = t.stride(0)
    assert getattr(ln.lib(), name)(args(names, layout, {}, **fields)) == g.OK


def inputs(dim, rows):
    q = torch.Generator(device="cuda")
    q.manual_seed(dim)
    pad = dim % 3
    return (lambda: strided(normal(q, (rows, dim), torch.bfloat16), pad, pad % 2),
            normal(q, (dim,), torch.bfloat16, 0.2) + 1)


def like(t):
    """A tensor of t's strides, NaN around it, with t's values."""
    return strided(t, t.stride(0) - t.shape[1], t.storage_offset())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dim", DIMS)
def test_h_in_an_inputs_memory(dim, eight):
    rows = 37
    make, w = inputs(dim, rows)
    x, res = make(), make()
    want = g.rms_norm(x, w, res, with_rstd=True,
                      out_dtype=torch.float8_e4m3fn if eight else None)
    for where in ("x", "residual"):
        t = {"x": like(x), "residual": like(res), "weight": w,
             "y": torch.empty((rows, -(-dim // 16) * 16), dtype=want.y.dtype, device="cuda")[:, :dim],
             "rstd": torch.empty(rows, device="cuda")}
        t["h"] = t[where]
        if eight:
            t["scale"] = torch.empty(rows, device="cuda")
        call("rms_norm_forward", NORM, NORM_STRUCT, t, rows=rows, dim=dim, type=BF16,
             out_type=E4M3 if eight else BF16, eps=1e-5)
        assert torch.equal(t["h"], want.h) and torch.equal(t["rstd"], want.rstd)
        assert torch.equal(t["y"].float(), want.y.float())
        other = "residual" if where == "x" else "x"
        assert torch.equal(t[other], {"x": x, "residual": res}[other])
        if eight:
            assert torch.equal(t["scale"], want.scale)


def test_h_in_xs_memory_without_a_residual():
    make, w = inputs(500, 5)
    x = make()
    want = g.rms_norm(x, w)
    t = {"x": like(x), "weight": w, "y": torch.empty((5, 500), dtype=x.dtype, device="cuda")}
    t["h"] = t["x"]
    call("rms_norm_forward", NORM, NORM_STRUCT, t, rows=5, dim=500, type=BF16, out_type=BF16,
         eps=1e-5)
    assert torch.equal(t["y"], want.y) and torch.equal(t["x"], x)


@pytest.mark.parametrize("rows", [1, 700])
@pytest.mark.parametrize("dim", DIMS)
def test_dx_in_an_inputs_memory(dim, rows):
    make, w = inputs(dim, rows)
    dy, dh, h = make(), make(), make()
    rstd = torch.rand(rows, device="cuda") + 0.5
    want = g.rms_norm_backward(dy, h, w, rstd, dh=dh)
    values = dict(rows=rows, dim=dim, type=BF16)
    for where in ("dy", "dh"):
        t = {"dy": like(dy), "dh": like(dh), "h": h, "weight": w, "rstd": rstd,
             "dweight": torch.empty(dim, dtype=w.dtype, device="cuda")}
        t["dx"] = t[where]
        ws = torch.empty((1024 * (dim + 32),), device="cuda")
        t["workspace"] = ws
        call("rms_norm_backward", NORM_BACKWARD, NORM_BACKWARD_STRUCT, t, **values,
             workspace_bytes=ws.numel() * 4)
        assert torch.equal(t["dx"], want[0]) and torch.equal(t["dweight"], want[1])
