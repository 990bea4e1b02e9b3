"""The layer norm and its backward pass on the GPU against their formulas in 64 bits.

Bounds (see linear_norm_util.py for the general ones).  In fp32, h is off by 2^-24 of itself.  The
mean is the first mean plus the mean of the differences c from it: off by the roundings of h and c,
at most 2^-23 of |h| and |mean| each on average, and by (dim + 16) 2^-23 of the mean of |c|.  A
difference is off by e_c = 2^-23 (|h| + |mean|) and the mean's error; the variance, relative to var +
eps, by (dim + 16) 2^-23 (its terms have one sign) and twice the mean of |c| e_c; rstd by half of
that.  In 8 bits half a step is 2^-4 of the value or 2^-10 scale (e4m3), scale / 2 (int8)."""
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


def inputs(q, rows, dim, dt, pad=0, residual=True, level=0.5):
    x = strided(normal(q, (rows, dim), dt, 0.5), pad, pad % 2)
    r = None
    if residual:
        r = normal(q, (rows, dim), torch.float32, 2.0) + level * normal(q, (rows, 1), torch.float32)
        r = strided(r.to(dt), pad, pad % 2)
    w = (1 + 0.2 * torch.randn(dim, generator=q, device="cuda")).to(dt)
    return x, r, w, normal(q, (dim,), dt, 0.3)


def ln64(x, r, w, b, eps=EPS):
    """(h, mean, rstd, y, bound of mean, relative bound of rstd, bound of y), the bounds of fp32."""
    dim = x.shape[1]
    h = x.double() + (0 if r is None else r.double())
    mean = h.mean(1, keepdim=True)
    c = h - mean
    var = c.square().mean(1, keepdim=True) + eps
    rstd = 1 / var.sqrt()
    y = c * rstd * w.double() + (0 if b is None else b.double())
    e_mean = F32 * (h.abs().mean(1, keepdim=True) + 2 * mean.abs()
                    + (dim + 16) * c.abs().mean(1, keepdim=True))
    e_c = F32 * (h.abs() + mean.abs()) + e_mean
    rel = (dim + 16) * F32 + (c.abs() * e_c + e_c.square()).mean(1, keepdim=True) / var
    e_y = w.double().abs() * rstd * (e_c + (c.abs() + e_c) * rel) + 4 * F32 * (
        (c * rstd * w.double()).abs() + y.abs())
    return h, mean[:, 0], rstd[:, 0], y, e_mean[:, 0], rel[:, 0], e_y


def check_stats(got, mean, rstd, e_mean, rel):
    assert bool(((got.mean.double() - mean).abs() <= e_mean).all())
    assert bool(((got.rstd.double() - rstd).abs() <= (rel + 4 * F32) * rstd).all())


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("dim", DIMS)
def test_norm(dim, ty):
    dt = DT[ty]
    rows = 1 + dim % 5
    for residual, bias in ((True, True), (False, False)):
        x, r, w, b = inputs(gen(dim), rows, dim, dt, dim % 4, residual)
        b = b if bias else None
        print(f"layer norm {rows}x{dim} {ty} residual {residual}", flush=True)
        got = g.layer_norm(x, w, b, r, eps=EPS, with_stats=True)
        h, mean, rstd, y, e_mean, rel, e_y = ln64(x, r, w, b)
        assert_close(got.y, y, e_y, "y")
        assert got.scale is None
        check_stats(got, mean, rstd, e_mean, rel)
        if residual:
            assert_close(got.h, h, F32 * h.abs(), "h")
        else:
            assert got.h is x
        assert torch.equal(g.layer_norm(x, w, b, r, eps=EPS).y, got.y)


@pytest.mark.parametrize("out", [E4M3, torch.int8])
@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("dim", DIMS)
def test_norm_in_8_bits(dim, ty, out):
    dt = DT[ty]
    rows = 1 + dim % 3
    x, r, w, b = inputs(gen(dim), rows, dim, dt, dim % 3)
    got = g.layer_norm(x, w, b, r, eps=EPS, out_dtype=out)
    h, _, _, y, _, _, e_y = ln64(x, r, w, b)
    top = 448 if out == E4M3 else 127
    scale = y.abs().amax(1) / top
    assert got.y.dtype == out and got.rstd is None and got.mean is None
    assert got.y.stride(0) % 16 == 0 or rows == 1
    assert_close(got.h, h, F32 * h.abs(), "h")
    e_scale = e_y.amax(1) / top + 2 * F32 * scale
    assert bool(((got.scale.double() - scale).abs() <= e_scale).all())
    back = got.y.double() * got.scale.double()[:, None]
    if out == E4M3:
        bound = (2.0 ** -4 + 4 * F32) * y.abs() + 2.0 ** -10 * scale[:, None] + 2 * e_y
    else:   # a quotient is off by 2^-23 of its value, 127 scales at most
        bound = (0.5 + 128 * F32) * got.scale.double()[:, None] + 2 * e_y
    assert bool(((back - y).abs() <= bound + top * e_scale[:, None]).all())


@pytest.mark.parametrize("out", [E4M3, torch.int8])
@pytest.mark.parametrize("dim", [1, 8, 100, 513, 1024, 3000, 8192, 20000])
def test_rms_norm_beside_it(dim, out):
    """The other norm's 8-bit rows: the scale is the row's, the values its quotients."""
    x, r, w, _ = inputs(gen(dim), 3, dim, torch.bfloat16)
    got = g.rms_norm(x, w, r, eps=EPS, out_dtype=out)
    h = x.double() + r.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w.double()
    rel, top = (dim + 20) * F32, 448 if out == E4M3 else 127
    scale = y.abs().amax(1) / top
    assert bool(((got.scale.double() - scale).abs() <= rel * scale).all())
    back = got.y.double() * got.scale.double()[:, None]
    step = (2.0 ** -4 * y.abs() + 2.0 ** -10 * scale[:, None] if out == E4M3
            else 0.5 * scale[:, None])
    assert bool(((back - y).abs() <= step + 3 * rel * (y.abs() + step)).all())


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("dim", [3, 1000, 4096, 20000])
def test_rows_far_from_zero(dim, ty):
    """Means of some hundred deviations: the deviation keeps its bits."""
    q, dt = gen(dim + 7), DT[ty]
    x = (normal(q, (4, dim), torch.float32) + torch.tensor([[300.0], [-200.0], [0.0], [100.0]],
                                                           device="cuda")).to(dt)
    w, b = torch.ones(dim, dtype=dt, device="cuda"), torch.zeros(dim, dtype=dt, device="cuda")
    got = g.layer_norm(x, w, b, eps=EPS, with_stats=True)
    h, mean, rstd, y, e_mean, rel, e_y = ln64(x, None, w, b)
    # h is exact here, and so are the differences from a mean within a factor of 2 of it: what is
    # left are (dim + 16) roundings of |c| and the mean's own
    c = (h - mean[:, None]).abs()
    e_mean = F32 * (2 * mean.abs() + (dim + 16) * c.mean(1))
    e_c = F32 * (c + mean[:, None].abs()) + e_mean[:, None]
    rel = (dim + 16) * F32 + (c * e_c + e_c.square()).mean(1) * rstd.square()
    check_stats(got, mean, rstd, e_mean, rel)
    assert_close(got.y, y, rstd[:, None] * (e_c + c * rel[:, None]) + 4 * F32 * y.abs())


def test_rows_of_zeros_nan_and_infinity():
    dim = 200
    q = gen(5)
    for dt in DT.values():
        x, r, w, b = inputs(q, 6, dim, dt)
        b[3] = 2.0
        x[0] = 0
        r[0] = 0
        x[1, 7] = float("nan")
        x[2, 9] = float("inf")
        for out in (None, E4M3, torch.int8):
            got = g.layer_norm(x, w, b, r, out_dtype=out, with_stats=True)
            y = got.y.double()
            if got.scale is not None:
                y = y * got.scale.double()[:, None]
            assert got.mean[0] == 0 and abs(got.rstd[0].item() - 1e5 ** 0.5) <= 1e-3
            assert bool(y[1:3].isnan().all()) and bool(got.rstd[1:3].isnan().all())
            # a row of zeros is the bias
            if out is None:
                assert torch.equal(got.y[0], b)
            assert bool(torch.isfinite(y[3:]).all()) and bool(torch.isfinite(y[0]).all())
        zero = g.layer_norm(x[:1], w, None, r[:1], out_dtype=torch.int8)
        assert zero.scale[0] == 1 and not zero.y.any()


def test_constant_rows():
    """All values alike: the deviation is 0, however far from 0 the row is."""
    for dim in (1, 5, 4096, 17000):
        x = torch.full((2, dim), 777.0, dtype=torch.bfloat16, device="cuda")
        w, b = torch.ones_like(x[0]), torch.full_like(x[0], 0.5)
        got = g.layer_norm(x, w, b, eps=1e-5, with_stats=True)
        # the mean of equal values is off by 2^-23 of it at most, the difference exact
        assert bool(((got.mean.double() - x[0, 0].double()).abs() <= 2 * F32 * 777).all())
        assert bool(((got.y.double() - 0.5).abs() <= 2 * F32 * 777 * 1e5 ** 0.5 + 2.0 ** -9).all())


@pytest.mark.parametrize("dim", [64, 1000, 8192, 20000])
def test_squares_outside_fp32(dim):
    q = gen(dim)
    w, b = torch.ones(dim, dtype=torch.bfloat16, device="cuda"), torch.zeros(
        dim, dtype=torch.bfloat16, device="cuda")
    for size, eps in ((1e30, 1e-5), (1e-25, 0.0), (2e37, 0.0)):
        x = (torch.randn((3, dim), generator=q, device="cuda") * size).bfloat16()
        got = g.layer_norm(x, w, b, eps=eps, with_stats=True)
        h, mean, rstd, y, e_mean, rel, e_y = ln64(x, None, w, b, eps)
        check_stats(got, mean, rstd, e_mean, rel)
        assert_close(got.y, y, e_y)


def test_no_rows():
    w = torch.ones(16, dtype=torch.float16, device="cuda")
    x = torch.empty((0, 16), dtype=torch.float16, device="cuda")
    got = g.layer_norm(x, w, w, x, out_dtype=torch.int8, with_stats=True)
    assert got.y.shape == (0, 16) and got.scale.shape == (0,) and got.mean.shape == (0,)
    dx, dw, db = g.layer_norm_backward(x, x, w, got.mean, got.rstd)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()


def ln_backward64(dy, h, w, mean, rstd, dh):
    dim = dy.shape[1]
    r = rstd.double()[:, None]
    c = h.double() - mean.double()[:, None]
    xh, gr = c * r, dy.double() * w.double()
    level, along = gr.mean(1, keepdim=True), (gr * xh).mean(1, keepdim=True)
    want = r * (gr - level - xh * along)
    # a difference is rounded once more, relative to itself
    err = (dim + 20) * F32 * r * (gr.abs() + gr.abs().mean(1, keepdim=True)
                                  + xh.abs() * (gr * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        want = want + dh.double()
        err = err + F32 * dh.double().abs()
    return want, err + F32 * want.abs(), dy.double() * xh


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("rows,dim", [(1 + 7 * i % 40, d) for i, d in enumerate(DIMS)]
                         + [(700, 96), (1500, 1000), (513, 4096), (600, 17000), (2, 16000)])
def test_backward(rows, dim, ty):
    dt = DT[ty]
    q = gen(rows + dim)
    pad = dim % 3
    h = strided((normal(q, (rows, dim), torch.float32, 2.0) + 1.5).to(dt), pad)
    dy = strided(normal(q, (rows, dim), dt), pad, 1)
    dh = strided(normal(q, (rows, dim), dt), pad) if dim % 2 else None
    w = (1 + 0.2 * torch.randn(dim, generator=q, device="cuda")).to(dt)
    mean = h.double().mean(1).float()
    rstd = (1 / ((h.double() - mean.double()[:, None]).square().mean(1) + EPS).sqrt()).float()
    print(f"layer norm backward {rows}x{dim} {ty}", flush=True)
    dx, dw, db = g.layer_norm_backward(dy, h, w, mean, rstd, dh=dh)
    want, err, t = ln_backward64(dy, h, w, mean, rstd, dh)
    assert_close(dx, want, err, "dx")
    assert_close(dw, t.sum(0), (rows + 16) * F32 * t.abs().sum(0), "dweight")
    assert_close(db, dy.double().sum(0), (rows + 16) * F32 * dy.double().abs().sum(0), "dbias")
    for weight_grad, bias_grad in ((True, False), (False, True), (False, False)):
        got = g.layer_norm_backward(dy, h, w, mean, rstd, dh=dh, weight_grad=weight_grad,
                                    bias_grad=bias_grad)
        assert torch.equal(got[0], dx)
        assert torch.equal(got[1], dw) if weight_grad else got[1] is None
        assert torch.equal(got[2], db) if bias_grad else got[2] is None


def test_backward_against_differences():
    """<gradient, u> against the central difference of the norm's 64-bit formula along u."""
    q = gen(21)
    dt = torch.float16
    rows, dim = 5, 96
    x, r, w, b = inputs(q, rows, dim, dt)
    dy, dh = normal(q, (rows, dim), dt), normal(q, (rows, dim), dt)
    got = g.layer_norm(x, w, b, r, eps=EPS, with_stats=True)
    grads = g.layer_norm_backward(dy, got.h, w, got.mean, got.rstd, dh=dh)

    def loss(x64, w64, b64):
        h, _, _, y, *_ = ln64(x64, r, w64, b64)
        return (y * dy.double()).sum() + (h * dh.double()).sum()

    for i, grad in enumerate(grads):
        z = [x.double(), w.double(), b.double()]
        u = torch.randn(z[i].shape, generator=q, device="cuda", dtype=torch.float64)
        lo, hi = list(z), list(z)
        lo[i], hi[i] = z[i] - 1e-4 * u, z[i] + 1e-4 * u
        want = ((loss(*hi) - loss(*lo)) / 2e-4).item()
        diff = abs((grad.double() * u).sum().item() - want)
        # h and the gradient are each rounded to 2^-11; terms are of magnitude up to about 4
        assert diff <= 4 * 2.0 ** -11 * ((grad.double().abs() + 4) * u.abs()).sum().item()


@pytest.mark.parametrize("dt", [E4M3, torch.int8])
def test_8_bit_norm_feeds_the_8_bit_layer(dt):
    """The norm's rows and scales go into linear as they are."""
    q = gen(22)
    for rows, dim, n in ((1, 200, 48), (16, 1000, 80), (100, 392, 130)):
        x, r, w, b = inputs(q, rows, dim, torch.bfloat16)
        wq = g.quantize_rows(normal(q, (n, dim), torch.bfloat16), dtype=dt)
        a = g.layer_norm(x, w, b, r, out_dtype=dt)
        got = g.linear(a.y, wq.values.t(), scale_a=a.scale, scale_b=wq.scale)
        a64 = a.y.double() * a.scale.double()[:, None]
        b64 = wq.values.double() * wq.scale.double()[:, None]
        want, mag = a64 @ b64.t().contiguous(), a64.abs() @ b64.t().abs().contiguous()
        assert_close(got, want, (dim + 16) * F32 * mag)


def test_graph_replays():
    q = gen(23)
    x, r, w, b = inputs(q, 300, 1000, torch.bfloat16)
    dy = normal(q, (300, 1000), torch.bfloat16)

    def step():
        n = g.layer_norm(x, w, b, r, with_stats=True)
        q8 = g.layer_norm(x, w, b, r, out_dtype=torch.int8)
        return (n.y, n.h, n.mean, n.rstd, q8.y, q8.scale,
                *g.layer_norm_backward(dy, n.h, w, n.mean, n.rstd, dh=dy))

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
        for a, c in zip(held, want):
            assert torch.equal(a, c), i
