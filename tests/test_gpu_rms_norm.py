"""The root-mean-square norm and its backward pass on the GPU against their formulas in 64 bits.

Bounds (see linear_norm_util.py for the general ones): a mean of dim squares in fp32 is off by
at most (dim + 8) 2^-23 of its value (all terms have one sign), rstd by half of that, y by that
and a few fp32 products; in 8 bits half a step is 2^-4 of the value, or 2^-10 scale below the
smallest normal number 2^-6."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import F32, assert_close, normal, strided  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
EPS = 1e-5
# one per row shape, its borders, odd sizes, and rows too long for registers
DIMS = [1, 2, 7, 8, 64, 511, 512, 513, 1024, 1025, 2048, 2055, 4093, 4096, 4097, 8192, 8199,
        16384, 16385, 20000, 33001]


def gen(seed):
    q = torch.Generator(device="cuda")
    q.manual_seed(seed)
    return q


def inputs(q, rows, dim, dt, pad=0, residual=True):
    x = strided(normal(q, (rows, dim), dt, 0.5), pad, pad % 2)
    r = strided(normal(q, (rows, dim), dt, 2.0), pad, pad % 2) if residual else None
    return x, r, (1 + 0.2 * torch.randn(dim, generator=q, device="cuda")).to(dt)


def norm64(x, r, w, eps=EPS):
    h = x.double() + (0 if r is None else r.double())
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w.double()


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("dim", DIMS)
def test_norm(dim, ty):
    dt = DT[ty]
    rows = 1 + dim % 5
    for residual in (True, False):
        x, r, w = inputs(gen(dim), rows, dim, dt, dim % 4, residual)
        print(f"norm {rows}x{dim} {ty} residual {residual}", flush=True)
        got = g.rms_norm(x, w, r, eps=EPS, with_rstd=True)
        h, rstd, y = norm64(x, r, w)
        rel = (dim + 16) * F32
        assert_close(got.y, y, rel * y.abs(), "y")
        assert got.scale is None
        assert bool(((got.rstd.double() - rstd).abs() <= rel * rstd).all())
        if residual:
            assert_close(got.h, h, F32 * h.abs(), "h")
        else:
            assert got.h is x


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("dim", DIMS)
def test_norm_in_8_bits(dim, ty):
    dt = DT[ty]
    rows = 1 + dim % 3
    x, r, w = inputs(gen(dim), rows, dim, dt, dim % 3)
    got = g.rms_norm(x, w, r, eps=EPS, out_dtype=E4M3)
    h, rstd, y = norm64(x, r, w)
    scale = y.abs().amax(1) / 448
    rel = (dim + 16) * F32
    assert got.y.dtype == E4M3 and got.rstd is None
    assert got.y.stride(0) % 16 == 0 or rows == 1
    assert_close(got.h, h, F32 * h.abs(), "h")
    assert bool(((got.scale.double() - scale).abs() <= rel * scale).all())
    back = got.y.double() * got.scale.double()[:, None]
    bound = (2.0 ** -4 + rel) * y.abs() + 2.0 ** -10 * scale[:, None]
    assert bool(((back - y).abs() <= bound).all())


def test_rows_of_zeros_nan_and_infinity():
    dim = 200
    q = gen(5)
    for dt in DT.values():
        x, r, w = inputs(q, 6, dim, dt)
        x[0] = 0
        r[0] = 0
        x[1, 7] = float("nan")
        x[2, 9] = float("inf")
        got = g.rms_norm(x, w, r, out_dtype=E4M3, with_rstd=True)
        assert got.scale[0] == 1 and not got.y[0].float().any() and not got.h[0].any()
        assert abs(got.rstd[0].item() - 1e5 ** 0.5) <= 1e-3
        assert got.scale[1] == 1 and bool(got.y[1].float().isnan().all())
        # h / inf is 0, inf / inf is NaN
        assert got.scale[2] == 1 and bool(got.y[2, 9].float().isnan()) and got.rstd[2] == 0
        assert bool(torch.isfinite(got.y[3:].float()).all())
        h, rstd, y = norm64(x[3:], r[3:], w)
        y16 = g.rms_norm(x, w, r).y
        assert_close(y16[3:], y, (dim + 16) * F32 * y.abs())
        assert bool(y16[1].isnan().all()) and not y16[0].any()


def test_tiny_rows_keep_a_finite_scale():
    """A row so small that its largest magnitude / 448 is below the smallest normal fp32."""
    x = torch.full((2, 64), 2.0 ** -130, dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    got = g.rms_norm(x, w, eps=1.0, out_dtype=E4M3)
    assert got.scale[0].item() == 2.0 ** -126 and bool(torch.isfinite(got.y.float()).all())


def test_no_rows():
    w = torch.ones(16, dtype=torch.float16, device="cuda")
    x = torch.empty((0, 16), dtype=torch.float16, device="cuda")
    got = g.rms_norm(x, w, x, out_dtype=E4M3, with_rstd=True)
    assert got.y.shape == (0, 16) and got.scale.shape == (0,) and got.rstd.shape == (0,)
    dx, dw = g.rms_norm_backward(x, x, w, got.rstd)
    assert dx.shape == (0, 16) and not dw.any()


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("rows,dim", [(1 + 7 * i % 40, d) for i, d in enumerate(DIMS)]
                         + [(700, 96), (1500, 1000), (513, 4096), (600, 17000)])
def test_backward(rows, dim, ty):
    dt = DT[ty]
    q = gen(rows + dim)
    pad = dim % 3
    h = strided(normal(q, (rows, dim), dt, 2.0), pad)
    dy = strided(normal(q, (rows, dim), dt), pad, 1)
    dh = strided(normal(q, (rows, dim), dt), pad) if dim % 2 else None
    w = (1 + 0.2 * torch.randn(dim, generator=q, device="cuda")).to(dt)
    rstd = (1 / (h.double().square().mean(1) + EPS).sqrt()).float()
    print(f"norm backward {rows}x{dim} {ty}", flush=True)
    dx, dw = g.rms_norm_backward(dy, h, w, rstd, dh=dh)
    r = rstd.double()[:, None]
    xh, gr = h.double() * r, dy.double() * w.double()
    want = r * (gr - xh * (gr * xh).mean(1, keepdim=True))
    err = (dim + 16) * F32 * r * (gr.abs() + xh.abs() * (gr * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        want = want + dh.double()
        err = err + F32 * dh.double().abs()
    assert_close(dx, want, err + F32 * want.abs(), "dx")
    t = dy.double() * xh
    assert_close(dw, t.sum(0), (rows + 16) * F32 * t.abs().sum(0), "dweight")
    assert g.rms_norm_backward(dy, h, w, rstd, dh=dh, weight_grad=False)[1] is None


def test_backward_against_differences():
    """<gradient, u> against the central difference of the norm's 64-bit formula along u."""
    q = gen(21)
    dt = torch.float16
    rows, dim = 5, 96
    x, r, w = inputs(q, rows, dim, dt)
    dy, dh = normal(q, (rows, dim), dt), normal(q, (rows, dim), dt)
    got = g.rms_norm(x, w, r, eps=EPS, with_rstd=True)
    dx, dw = g.rms_norm_backward(dy, got.h, w, got.rstd, dh=dh)

    def loss(x64, w64):
        h, _, y = norm64(x64, r, w64)
        return (y * dy.double()).sum() + (h * dh.double()).sum()

    for i, grad in enumerate((dx, dw)):
        z = [x.double(), w.double()]
        u = torch.randn(z[i].shape, generator=q, device="cuda", dtype=torch.float64)
        lo, hi = list(z), list(z)
        lo[i], hi[i] = z[i] - 1e-4 * u, z[i] + 1e-4 * u
        want = ((loss(*hi) - loss(*lo)) / 2e-4).item()
        diff = abs((grad.double() * u).sum().item() - want)
        # h and the gradient are each rounded to 2^-11; terms are of magnitude up to about 4
        assert diff <= 4 * 2.0 ** -11 * ((grad.double().abs() + 4) * u.abs()).sum().item()


def test_8_bit_norm_feeds_the_8_bit_layer():
    """The norm's rows and scales go into linear as they are."""
    q = gen(22)
    for rows, dim, n in ((1, 200, 48), (100, 392, 130)):
        x, r, w = inputs(q, rows, dim, torch.bfloat16)
        wt, sw = g_e4m3(torch.randn((n, dim), generator=q, device="cuda"))
        a = g.rms_norm(x, w, r, out_dtype=E4M3)
        got = g.linear(a.y, wt.t(), scale_a=a.scale, scale_b=sw)
        a64 = a.y.double() * a.scale.double()[:, None]
        b64 = wt.double() * sw.double()[:, None]
        want, mag = a64 @ b64.t().contiguous(), a64.abs() @ b64.t().abs().contiguous()
        assert_close(got, want, (dim + 16) * F32 * mag)


def g_e4m3(v):
    from linear_norm_util import e4m3_rows
    return e4m3_rows(v)


def test_graph_replays():
    q = gen(23)
    x, r, w = inputs(q, 300, 1000, torch.bfloat16)
    dy = normal(q, (300, 1000), torch.bfloat16)

    def step():
        n = g.rms_norm(x, w, r, with_rstd=True)
        q8 = g.rms_norm(x, w, r, out_dtype=E4M3)
        return (n.y, n.h, n.rstd, q8.y.float(), q8.scale,
                *g.rms_norm_backward(dy, n.h, w, n.rstd, dh=dy))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        x.copy_(normal(q, (300, 1000), torch.bfloat16))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b), i
