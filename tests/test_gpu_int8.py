"""The linear layer on int8 operands, and rows quantised for it, on the GPU.

Sums are exact in 32-bit integers, so a result differs from the definition's by the fp32 roundings
after them (the sum's own, two scales, bias: 2^-24 each of what they round), the activation's 2^-20
and the last one to 16 bits.  With sums below 2^24, scales that are powers of two and whole-numbered
bias and residual there is only the last, and results are equal bit for bit."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import F32, act, assert_close, mm, normal, strided  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# few rows (in one piece, in slices of k, wide), 64 x 64 tiles, 128 x 128, 256 x 256, slivers
SIZES = [(1, 16, 16), (1, 33, 129), (1, 1, 1), (2, 7, 15), (3, 100, 1000), (16, 256, 128),
         (16, 17, 5000), (9, 40, 8000), (16, 8192, 4096), (12, 16400, 130), (17, 64, 127),
         (64, 64, 128), (100, 200, 300), (70, 90, 4999), (40, 70, 16000), (1900, 2050, 260),
         (2048, 2048, 256), (1100, 1000, 4098), (3600, 3650, 391), (3584, 3840, 640),
         (4097, 4100, 257), (300, 8192, 2050)]


def gen(seed):
    q = torch.Generator(device="cuda")
    q.manual_seed(seed)
    return q


def rows8(v, pad=0):
    """v (whole numbers) as int8 rows on 16-byte boundaries, 77 in what lies between."""
    x, k = v.shape
    buf = torch.full((x, -(-k // 16) * 16 + 16 * pad), 77, dtype=torch.int8, device="cuda")
    buf[:, :k] = v.to(torch.int8)
    return buf[:, :k]


def whole(q, shape, top):
    return torch.randint(-top, top + 1, shape, generator=q, device="cuda").float()


@pytest.mark.parametrize("m,n,k", SIZES)
def test_values(m, n, k):
    q, dt = gen(m + n + k), (torch.bfloat16 if m % 2 else torch.float16)
    a, w = rows8(whole(q, (m, k), 127), m % 2), rows8(whole(q, (n, k), 127), n % 2)
    sa = torch.rand(m, generator=q, device="cuda") * 0.02 + 1e-3
    sb = (torch.rand(n, generator=q, device="cuda") * 0.02 + 1e-3) * k ** -0.5
    bias = normal(q, (n,), dt) if n % 2 else None
    res = strided(normal(q, (m, n), dt), m % 3) if m > 2 else None
    activation = ACTS[(n + k) % 5]
    print(f"int8 {m}x{n}x{k} {activation}", flush=True)
    got = g.linear(a, w.t(), bias, res, activation=activation, scale_a=sa, scale_b=sb,
                   out_dtype=dt, with_pre=k % 2 == 0)
    v = mm(a.double(), w.double().t()) * sa.double()[:, None] * sb.double()[None, :]
    err = 3 * F32 * v.abs()
    if bias is not None:
        v = v + bias.double()
        err = err + F32 * (v.abs() + bias.double().abs())
    if k % 2 == 0:
        assert_close(got[1], v, err, "pre")
        got = got[0]
    want, oerr = act(v, activation), 1.13 * err
    if activation not in ("none", "relu"):
        oerr = oerr + 2.0 ** -20 * v.abs()
    if res is not None:
        want = want + res.double()
        oerr = oerr + F32 * (want.abs() + res.double().abs())
    assert got.shape == (m, n) and got.dtype == dt
    assert_close(got, want, oerr, "out")


@pytest.mark.parametrize("out", DT)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_whole_numbers_bit_for_bit(m, n, k, out):
    """Products of up to 9 in magnitude: sums stay below 2^24."""
    q, dt = gen(m * 3 + n + k), DT[out]
    a, w = rows8(whole(q, (m, k), 3), 1), rows8(whole(q, (n, k), 3))
    sa = 2.0 ** whole(q, (m,), 1)
    sb = torch.full((n,), 0.5, device="cuda")
    bias, res = whole(q, (n,), 8).to(dt), whole(q, (m, n), 8).to(dt)
    got = g.linear(a, w.t(), bias, res, scale_a=sa, scale_b=sb, out_dtype=dt, activation="relu")
    v = mm(a.double(), w.double().t()) * (0.5 * sa.double()[:, None]) + bias.double()
    want = v.clamp(min=0) + res.double()
    assert torch.equal(got, want.float().to(dt))


@pytest.mark.parametrize("m,n", [(1, 16), (3, 33), (20, 40), (130, 70)])
def test_the_largest_sums(m, n):
    """k = 131071 values of -128: 2^31 - 2^14 is the largest sum that 32 bits hold."""
    k = 131071
    a = torch.full((m, k + 1), -128, dtype=torch.int8, device="cuda")[:, :k]
    w = torch.full((n, k + 1), -128, dtype=torch.int8, device="cuda")[:, :k]
    w[0] = 127
    sa = torch.full((m,), 2.0 ** -31, device="cuda")
    got = g.linear(a, w.t(), scale_a=sa, out_dtype=torch.float16)
    # 2^31 - 2^14 is a number of fp32
    want = torch.full((m, n), k * 2.0 ** 14, dtype=torch.float64, device="cuda")
    want[:, 0] = -k * 128 * 127
    assert torch.equal(got, (want.float() * 2.0 ** -31).half())


def test_one_deeper_is_refused():
    a = torch.zeros((2, 131072), dtype=torch.int8, device="cuda")
    with pytest.raises(g.GemmError) as e:
        g.linear(a, a.t())
    assert e.value.code == g.ERR_TOO_LARGE


def test_scales_are_optional_and_rows_with_nan_stay_alone():
    q = gen(6)
    for m, n, k in ((5, 40, 70), (90, 100, 70)):
        a, w = rows8(whole(q, (m, k), 5)), rows8(whole(q, (n, k), 5))
        plain = g.linear(a, w.t())
        assert plain.dtype == torch.bfloat16
        assert torch.equal(plain, mm(a.double(), w.double().t()).float().bfloat16())
        sa, sb = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
        sa[2], sb[7] = float("nan"), float("nan")
        bad = g.linear(a, w.t(), scale_a=sa, scale_b=sb).isnan()
        want = torch.zeros_like(bad)
        want[2], want[:, 7] = True, True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("m,n", [(0, 8), (8, 0), (3, 5), (70, 70)])
def test_empty_sizes(m, n):
    a = torch.empty((m, 0), dtype=torch.int8, device="cuda")
    b = torch.empty((0, n), dtype=torch.int8, device="cuda")
    q = gen(3)
    bias, res = normal(q, (n,), torch.float16), normal(q, (m, n), torch.float16)
    got = g.linear(a, b, bias, res, activation="relu", out_dtype=torch.float16)
    assert got.shape == (m, n)
    if m and n:
        assert_close(got, bias.double().clamp(min=0) + res.double(), F32 * 4)


# ---- rows quantised ----------------------------------------------------------------------------

def quantized(x, top):
    """(scales in fp32, quotients in 64 bits) of the definition."""
    amax = x.float().abs().amax(1)
    # rounded once: torch divides by a number with its rounded reciprocal
    scale = torch.where(amax > 0, (amax.double() / top).float(), torch.ones_like(amax))
    return scale, x.double() / scale.double()[:, None]


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("dim", [1, 3, 8, 100, 512, 513, 1024, 2047, 4096, 5000, 8192, 16384, 16385,
                                 33001])
def test_quantize_rows(dim, ty):
    q, dt = gen(dim), DT[ty]
    x = strided(normal(q, (1 + dim % 4, dim), dt, 3.0), dim % 3, dim % 2)
    for kind, top in ((torch.int8, 127), (torch.float8_e4m3fn, 448)):
        got = g.quantize_rows(x, dtype=kind)
        scale, want = quantized(x, top)
        assert got.values.dtype == kind and got.values.shape == x.shape
        assert got.values.stride(0) % 16 == 0 or x.shape[0] == 1
        assert torch.equal(got.scale, scale)
        off = (got.values.double() - want).abs()
        if kind == torch.int8:
            # a quotient in fp32 is off by 2^-23 of its value, and then rounded
            assert bool((off <= 0.5 + 127 * F32).all()) and int(got.values.int().abs().max()) <= 127
        else:
            assert bool((off <= 2.0 ** -4 * want.abs() * (1 + 16 * F32) + 2.0 ** -10).all())


def test_quantize_rows_of_zeros_nan_and_infinity():
    for dt in DT.values():
        x = normal(gen(1), (5, 300), dt)
        x[0] = 0
        x[1, 5] = float("nan")
        x[2, 6] = float("-inf")
        x[3] = torch.finfo(dt).smallest_normal
        got = g.quantize_rows(x)
        assert got.scale[0] == 1 and not got.values[0].any()
        assert bool(got.scale[1:3].isnan().all())
        assert bool(torch.isfinite(got.scale[3:]).all()) and bool(torch.isfinite(got.scale[:1]).all())
        assert int(got.values[4].int().abs().max()) == 127
        w = rows8(torch.ones((4, 300), device="cuda"))
        out = g.linear(got.values, w.t(), scale_a=got.scale)
        assert bool(out[1:3].isnan().all()) and bool(torch.isfinite(out[[0, 3, 4]]).all())


def test_quantized_rows_go_into_the_layer():
    """An output projection of 16-bit activations: within the two operands' half steps."""
    q = gen(8)
    for m, n, k in ((1, 100, 700), (50, 130, 700)):
        x, w = normal(q, (m, k), torch.bfloat16), normal(q, (n, k), torch.bfloat16, k ** -0.5)
        a, b = g.quantize_rows(x), g.quantize_rows(w)
        got = g.linear(a.values, b.values.t(), scale_a=a.scale, scale_b=b.scale)
        ea, eb = 0.51 * a.scale.double()[:, None], 0.51 * b.scale.double()[:, None]
        x64, w64 = x.double(), w.double()
        want = mm(x64, w64.t())
        err = mm(ea.expand_as(x64), w64.abs().t()) + mm(x64.abs() + ea, eb.expand_as(w64).t())
        assert_close(got, want, err)


def test_another_stream_and_graph_replays():
    q = gen(9)
    x, w = normal(q, (40, 500), torch.float16), g.quantize_rows(normal(q, (90, 500), torch.float16))

    def step(stream=None):
        a = g.quantize_rows(x, stream=stream)
        return a.values, a.scale, g.linear(a.values, w.values.t(), scale_a=a.scale,
                                           scale_b=w.scale, stream=stream)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    torch.cuda.current_stream().wait_stream(s)
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(4):
        x.copy_(normal(q, (40, 500), torch.float16))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for u, v in zip(held, want):
            assert torch.equal(u, v)
