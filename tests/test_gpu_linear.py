"""The linear layer and its backward pass on the GPU against their formulas in 64 bits: every
kernel path (few rows, each tile, split k), both storage orders of both operands, odd sizes and
strides, NaN in everything that lies around the operands.  Bounds: linear_norm_util.py."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import (F32, act, assert_close, e4m3_rows, half_step, linear64, mm,  # noqa: E402
                              normal, slope, strided)

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    q = torch.Generator(device="cuda")
    q.manual_seed(seed)
    return q


def operand(q, rows, cols, dtype, order, pad, offset, std=1.0):
    t = normal(q, (rows, cols) if order == "r" else (cols, rows), dtype, std)
    return strided(t if order == "r" else t.t(), pad, offset)


def check(m, n, k, ty, ao="r", bo="c", activation="none", bias=False, residual=False,
          with_pre=False, pad=0, offset=0, seed=1):
    dt = DT[ty]
    q = gen(seed)
    a = operand(q, m, k, dt, ao, pad, offset)
    b = operand(q, k, n, dt, bo, pad, offset, max(k, 1) ** -0.5)
    bi = normal(q, (n,), dt, 0.5) if bias else None
    r = strided(normal(q, (m, n), dt), pad, offset) if residual else None
    what = f"{m}x{n}x{k} {ty} {ao}{bo} {activation} pad {pad}"
    print(what, flush=True)
    got = g.linear(a, b, bi, r, activation=activation, with_pre=with_pre)
    out, pre, perr, oerr = linear64(a, b, bi, r, activation)
    if with_pre:
        assert_close(got[1], pre, perr, what + " pre")
        got = got[0]
    assert got.shape == (m, n) and got.dtype == dt
    assert_close(got, out, oerr, what)


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("bo", "rc")
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17])
@pytest.mark.parametrize("n,k", [(1, 1), (7, 31), (16, 64), (130, 257), (1000, 1030)])
def test_few_rows(m, n, k, bo, ty):
    check(m, n, k, ty, "r", bo, ACTS[(m + n) % 5], bias=n % 2 == 0, residual=m % 2 == 1,
          with_pre=k % 2 == 1, pad=m % 3, offset=m % 2, seed=m + n)


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("ao", "rc")
@pytest.mark.parametrize("bo", "rc")
@pytest.mark.parametrize("m,n,k", [(33, 65, 63), (64, 64, 64), (65, 130, 129), (200, 72, 200),
                                   (17, 300, 8), (257, 255, 511)])
def test_small_tiles(m, n, k, ao, bo, ty):
    check(m, n, k, ty, ao, bo, ACTS[(m + k) % 5], bias=True, residual=m % 2 == 0,
          with_pre=m % 2 == 1, pad=k % 2, offset=n % 2, seed=m * 3 + n)


@pytest.mark.parametrize("ao,bo", ["rr", "rc", "cr", "cc"])
@pytest.mark.parametrize("m,n,k,ty", [(1900, 2050, 200, "f16"), (2048, 1920, 128, "bf16"),
                                      (1801, 1999, 65, "bf16")])
def test_middle_tiles(m, n, k, ty, ao, bo):
    check(m, n, k, ty, ao, bo, "silu", bias=True, residual=True, with_pre=True, pad=m % 2,
          seed=m)


@pytest.mark.parametrize("ao,bo", ["rr", "rc", "cr", "cc"])
@pytest.mark.parametrize("m,n,k,ty", [(3600, 3650, 64, "f16"), (3841, 3583, 447, "bf16"),
                                      (3584, 3840, 385, "f16"), (4096, 3584, 40, "bf16")])
def test_large_tiles(m, n, k, ty, ao, bo):
    check(m, n, k, ty, ao, bo, "gelu_tanh", bias=True, residual=True, with_pre=m % 2 == 0,
          pad=n % 2, seed=n)


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("ao,bo", ["rr", "rc", "cr", "cc"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 8000), (5, 24, 6001), (40, 70, 5000), (100, 300, 4097)])
def test_split_k(m, n, k, ao, bo, ty):
    check(m, n, k, ty, ao, bo, "gelu", bias=True, residual=True, with_pre=True, seed=k)


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("ty", DT)
def test_activations(ty, activation):
    """Values from -12 to 12 through every activation: a (one column) times b (ones)."""
    dt = DT[ty]
    a = torch.linspace(-12, 12, 777, device="cuda").to(dt)[:, None]
    b = torch.ones((1, 24), dtype=dt, device="cuda")
    got = g.linear(a, b, activation=activation)
    out, _, _, oerr = linear64(a, b, None, None, activation)
    assert_close(got, out, oerr, f"{activation} {ty}")


@pytest.mark.parametrize("m,n", [(0, 8), (8, 0), (3, 5), (70, 70)])
def test_empty_sizes(m, n):
    """k = 0 leaves act(bias) + residual; m or n = 0 an empty result."""
    q = gen(3)
    a = torch.empty((m, 0), dtype=torch.float16, device="cuda")
    b = torch.empty((0, n), dtype=torch.float16, device="cuda")
    bias, res = normal(q, (n,), torch.float16), normal(q, (m, n), torch.float16)
    got = g.linear(a, b, bias, res, activation="silu")
    assert got.shape == (m, n)
    if m and n:
        want = act(bias.double(), "silu") + res.double()
        assert_close(got, want, 2.0 ** -19 * (1 + want.abs()), "k = 0")


def test_outside_values_stay_outside():
    """Infinities and NaN in one row and one column reach that row and column alone."""
    q = gen(4)
    for m, n, k in ((5, 40, 70), (90, 100, 70)):
        a, b = normal(q, (m, k), torch.bfloat16), normal(q, (k, n), torch.bfloat16)
        a[2, 3] = float("inf")
        b[5, 7] = float("nan")
        for bb in (b, b.t().contiguous().t()):
            got = g.linear(a, bb)
            bad = ~torch.isfinite(got)
            want = torch.zeros_like(bad)
            want[2, :] = True
            want[:, 7] = True
            assert torch.equal(bad, want)


def check8(m, n, k, out="bf16", activation="none", bias=False, residual=False, with_pre=False,
           scales=True, seed=1):
    q = gen(seed)
    dt = DT[out]
    a, sa = e4m3_rows(torch.randn((m, k), generator=q, device="cuda"))
    w, sb = e4m3_rows(torch.randn((n, k), generator=q, device="cuda"))
    if not scales:
        sa = sb = None
        a, w = (a.float() / 64).to(a.dtype), (w.float() / 64).to(w.dtype)
        a, w = (strided8(t) for t in (a, w))
    bi = normal(q, (n,), dt) if bias else None
    r = normal(q, (m, n), dt) if residual else None
    what = f"8-bit {m}x{n}x{k} {out} {activation}"
    print(what, flush=True)
    got = g.linear(a, w.t(), bi, r, activation=activation, scale_a=sa, scale_b=sb, out_dtype=dt,
                   with_pre=with_pre)
    o, pre, perr, oerr = linear64(a, w.t(), bi, r, activation, sa, sb)
    if with_pre:
        assert_close(got[1], pre, perr + 4 * F32 * pre.abs(), what + " pre")
        got = got[0]
    # the scales' two products in fp32
    assert_close(got, o, oerr + 4 * F32 * 1.13 * pre.abs(), what)


def strided8(t):
    buf = torch.full((t.shape[0], -(-t.shape[1] // 16) * 16 + 16), float("nan"),
                     device=t.device).to(t.dtype)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (1, 33, 129), (3, 100, 1000), (16, 256, 128),
                                   (16, 17, 5000), (17, 64, 127), (64, 64, 128), (100, 200, 300),
                                   (70, 90, 4999), (1900, 2050, 260), (2048, 2048, 256),
                                   (3600, 3650, 391), (3584, 3840, 640)])
def test_8_bit_operands(m, n, k):
    check8(m, n, k, "bf16" if m % 2 else "f16", ACTS[n % 5], bias=True, residual=m > 2,
           with_pre=k % 2 == 0, scales=m != 3, seed=k)


@pytest.mark.parametrize("m,n,k", [(5, 70, 64), (100, 90, 64), (9, 40, 8000)])
def test_result_in_the_residuals_memory(m, n, k):
    q = gen(9)
    a, b = normal(q, (m, k), torch.float16), normal(q, (k, n), torch.float16, 0.1)
    res = normal(q, (m, n), torch.float16)
    want = g.linear(a, b, residual=res)
    got = g.linear(a, b, residual=res, out=res)
    assert got is res and torch.equal(got, want)


def test_out_keeps_its_padding():
    q = gen(10)
    for m, n, k in ((3, 21, 40), (130, 77, 40)):
        a, b = normal(q, (m, k), torch.bfloat16), normal(q, (k, n), torch.bfloat16)
        buf = torch.full((m, n + 5), 7.0, dtype=torch.bfloat16, device="cuda")
        g.linear(a, b, out=buf[:, :n])
        assert bool((buf[:, n:] == 7.0).all()) and torch.equal(buf[:, :n], g.linear(a, b))


# ---- backward -----------------------------------------------------------------------------------

def check_backward(m, n, k, ty, ao="r", bo="c", activation="none", bias=True, pad=0, seed=1):
    dt = DT[ty]
    q = gen(seed)
    a = operand(q, m, k, dt, ao, pad, pad % 2)
    b = operand(q, k, n, dt, bo, pad, pad % 2, max(k, 1) ** -0.5)
    dc = strided(normal(q, (m, n), dt), pad)
    pre = strided(normal(q, (m, n), dt, 2.0), pad) if activation != "none" else None
    what = f"backward {m}x{n}x{k} {ty} {ao}{bo} {activation}"
    print(what, flush=True)
    da, db, dbias = g.linear_backward(dc, a, b, pre, activation=activation, bias_grad=bias)
    d, derr = dc.double(), 0.0 * dc.double()
    if pre is not None:
        d = d * slope(pre.double(), activation)
        derr = 2.0 ** -20 * (1 + pre.double().abs()) * dc.double().abs()
    # dpre is rounded once to the operands' type before it enters the products
    rerr = derr + half_step(dt) * d.abs() + 2.0 ** -25 if pre is not None else derr
    a64, b64 = a.double(), b.double()
    mag = d.abs() + rerr
    assert_close(da, mm(d, b64.t()),
                 mm(rerr, b64.abs().t()) + (n + 8) * F32 * mm(mag, b64.abs().t()), what + " da")
    assert_close(db, mm(a64.t(), d),
                 mm(a64.abs().t(), rerr) + (m + 8) * F32 * mm(a64.abs().t(), mag), what + " db")
    if bias:
        assert_close(dbias, d.sum(0), derr.sum(0) + (m + 8) * F32 * mag.sum(0), what + " dbias")
    else:
        assert dbias is None


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("ao,bo", ["rr", "rc", "cr", "cc"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 70, 33), (5, 64, 64), (70, 17, 129),
                                   (130, 200, 90), (513, 1025, 31)])
def test_backward(m, n, k, ao, bo, ty):
    check_backward(m, n, k, ty, ao, bo, ACTS[(m + n + k) % 5], bias=n % 2 == 0, pad=m % 3,
                   seed=m + k)


@pytest.mark.parametrize("activation", ACTS)
def test_backward_activations(activation):
    check_backward(100, 72, 40, "f16", "r", "c", activation, seed=2)


@pytest.mark.parametrize("m,n,k,ty", [(2100, 1900, 200, "bf16"), (3700, 300, 3650, "f16"),
                                      (300, 3700, 3650, "bf16"), (6000, 100, 130, "f16")])
def test_backward_large(m, n, k, ty):
    check_backward(m, n, k, ty, "r", "c", "gelu_tanh", seed=m)
    check_backward(m, n, k, ty, "r", "r", "none", seed=n)


def test_backward_parts_and_empty_sizes():
    q = gen(12)
    a, b = normal(q, (6, 10), torch.float16), normal(q, (10, 14), torch.float16)
    dc = normal(q, (6, 14), torch.float16)
    da, db, dbias = g.linear_backward(dc, a, b, bias_grad=True)
    assert torch.equal(g.linear_backward(dc, a, b, b_grad=False)[0], da)
    assert torch.equal(g.linear_backward(dc, a, b, a_grad=False)[1], db)
    assert g.linear_backward(dc, a, b, a_grad=False, b_grad=False) == (None, None, None)
    for m, n, k in ((0, 14, 10), (6, 0, 10), (6, 14, 0)):
        da, db, dbias = g.linear_backward(dc[:m, :n].contiguous(), a[:m, :k].contiguous(),
                                          b[:k, :n].contiguous(), bias_grad=True)
        assert da.shape == (m, k) and db.shape == (k, n) and dbias.shape == (n,)
        assert not da.any() if n == 0 else True
        assert not db.any() and not dbias.any() if m == 0 else True


@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu"])
def test_backward_against_differences(activation):
    """<gradient, u> against the central difference of the layer's 64-bit formula along u: the
    difference's own error is of order step^2."""
    q = gen(13)
    dt = torch.float16
    m, n, k = 20, 24, 18
    a, b = normal(q, (m, k), dt, 0.5), normal(q, (k, n), dt, 0.5)
    bias, dc = normal(q, (n,), dt, 0.5), normal(q, (m, n), dt)
    _, pre = g.linear(a, b, bias, activation=activation, with_pre=True)
    grads = g.linear_backward(dc, a, b, pre, activation=activation, bias_grad=True)

    def loss(a64, b64, bias64):
        return (act(mm(a64, b64) + bias64, activation) * dc.double()).sum()

    x = [t.double() for t in (a, b, bias)]
    for i, grad in enumerate(grads):
        u = torch.randn(x[i].shape, generator=q, device="cuda", dtype=torch.float64)
        lo, hi = list(x), list(x)
        lo[i], hi[i] = x[i] - 1e-4 * u, x[i] + 1e-4 * u
        want = ((loss(*hi) - loss(*lo)) / 2e-4).item()
        got = (grad.double() * u).sum().item()
        # every gradient element is a sum of at most 24 products of magnitude up to about 4, with
        # pre, dpre and the result rounded to 2^-11; the pairing with u averages over elements
        scale = (grad.double().abs() * u.abs()).sum().item() + 24 * u.abs().sum().item()
        assert abs(got - want) <= 4 * 2.0 ** -11 * scale


# ---- streams and graphs -------------------------------------------------------------------------

def test_given_stream():
    q = gen(14)
    a, b = normal(q, (40, 5000), torch.bfloat16), normal(q, (5000, 60), torch.bfloat16)
    want = g.linear(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = g.linear(a, b, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_graph_replays():
    """Forward and backward captured, replayed between eager calls on other values."""
    q = gen(15)
    m, n, k = 48, 80, 4100
    a, b = normal(q, (m, k), torch.float16), normal(q, (k, n), torch.float16, 0.02)
    bias = normal(q, (n,), torch.float16)

    def step():
        out, pre = g.linear(a, b, bias, activation="silu", with_pre=True)
        return (out, *g.linear_backward(out, a, b, pre, activation="silu", bias_grad=True))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        a.copy_(normal(q, (m, k), torch.float16))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for x, y in zip(held, want):
            assert torch.equal(x, y), i


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("bo", "rc")
@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (3, 9, 200), (64, 64, 64), (65, 127, 8), (200, 250, 70),
                                   (256, 256, 300), (255, 249, 61), (7, 200, 1000)])
def test_backward_in_one_launch(m, n, k, bo, ty):
    """Passes small enough for the kernel that makes dpre on the way (few panels, n and k of at
    least 8), every activation, with and without a bias gradient."""
    for i, activation in enumerate(ACTS):
        check_backward(m, n, k, ty, "r", bo, activation, bias=i % 3 != 1, pad=i % 3, seed=m + i)


def test_backward_in_one_launch_keeps_nan_in_its_row_and_column():
    """NaN in dc[i, j] reaches row i of da and column j of db and dbias, and nothing else."""
    q = gen(31)
    for bo in "rc":
        a = normal(q, (90, 40), torch.bfloat16)
        b = operand(q, 40, 70, torch.bfloat16, bo, 0, 0)
        dc, pre = normal(q, (90, 70), torch.bfloat16), normal(q, (90, 70), torch.bfloat16)
        dc[89, 3] = float("nan")
        da, db, dbias = g.linear_backward(dc, a, b, pre, activation="silu", bias_grad=True)
        rows, cols = da.isnan(), db.isnan()
        assert bool(rows[89].all()) and int(rows.sum()) == 40
        assert bool(cols[:, 3].all()) and int(cols.sum()) == 40
        assert bool(dbias[3].isnan()) and int(dbias.isnan().sum()) == 1


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("bo", "rc")
@pytest.mark.parametrize("n", [1, 3, 4, 5, 7, 61, 67, 130])
@pytest.mark.parametrize("k", [1, 5, 7, 8, 9, 33, 63, 449, 519, 1025, 2047])
def test_few_rows_at_every_edge(n, k, bo, ty):
    """Row ends inside a chunk, a unit and a batch of units; NaN lies right after every row."""
    for m in (1, 6, 16):
        check(m, n, k, ty, "r", bo, "relu", bias=True, pad=1 + m % 2, offset=k % 2, seed=n + k)


@pytest.mark.parametrize("n", [1, 15, 16, 70])
@pytest.mark.parametrize("k", [1, 7, 15, 16, 17, 31, 100, 129, 1000, 1039, 4097])
def test_few_rows_in_8_bits_at_every_edge(n, k):
    for m in (1, 9):
        check8(m, n, k, "f16", bias=True, seed=n + k)


@pytest.mark.parametrize("m,n", [(17, 70), (200, 130), (2100, 2050)])
@pytest.mark.parametrize("k", [1, 16, 40, 130, 512])
def test_short_8_bit_sums_are_exact_to_fp32(m, n, k):
    """The residual takes the rounded result away, so that the sum's own error shows: (k + 8)
    2^-23 of the products' magnitudes, and 2^-11 of what is left."""
    q = gen(k)
    a, sa = e4m3_rows(torch.randn((m, k), generator=q, device="cuda"))
    w, sb = e4m3_rows(torch.randn((n, k), generator=q, device="cuda"))
    kw = dict(scale_a=sa, scale_b=sb, out_dtype=torch.float16)
    first = g.linear(a, w.t(), **kw)
    rest = g.linear(a, w.t(), residual=-first, **kw)
    _, v, err, _ = linear64(a, w.t(), None, None, "none", sa, sb)
    left = rest.double() - (v - first.double())
    bound = err + 6 * F32 * v.abs() + half_step(torch.float16) * rest.double().abs() + 2.0 ** -25
    assert bool((left.abs() <= bound).all())
