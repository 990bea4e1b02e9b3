"""Results of at most 16 columns and slivers of as many past the last whole tile: a pass over a with
the operands exchanged, where both are k-contiguous.  Bounds: linear_norm_util.py; whole numbers bit
for bit; NaN around the operands and behind the results' rows."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import assert_close, linear64, mm, normal, strided  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
SIZES = [(17, 1, 8), (17, 16, 16), (40, 3, 31), (64, 8, 512), (100, 9, 1000), (257, 15, 513),
         (1000, 16, 4097), (4095, 1, 200), (3000, 17, 100), (2047, 1025, 130), (4100, 264, 96),
         (513, 4097, 300), (300, 2064, 257)]


def gen(seed):
    q = torch.Generator(device="cuda")
    q.manual_seed(seed)
    return q


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_forward(m, n, k, ty):
    dt, q, pad = DT[ty], gen(m + n + k), m % 3
    a = strided(normal(q, (m, k), dt), pad, pad % 2)
    b = strided(normal(q, (n, k), dt, k ** -0.5), pad).t()
    bias, res = normal(q, (n,), dt, 0.5), strided(normal(q, (m, n), dt), pad)
    activation = ACTS[(m + k) % 5]
    print(f"narrow {m}x{n}x{k} {ty} {activation}", flush=True)
    buf = torch.full((m, n + 5), 7.0, dtype=dt, device="cuda")
    _, pre = g.linear(a, b, bias, res, activation=activation, with_pre=True, out=buf[:, :n])
    out, pre64, perr, oerr = linear64(a, b, bias, res, activation)
    assert_close(pre, pre64, perr, "pre")
    assert_close(buf[:, :n], out, oerr, "out")
    assert bool((buf[:, n:] == 7.0).all())


@pytest.mark.parametrize("kind", ["f16", "bf16", "int8", "e4m3"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_whole_numbers_bit_for_bit(m, n, k, kind):
    """Operands of 1 and -1; the value before the activation packed as well."""
    q = gen(m * 3 + n + k)
    dt = DT.get(kind, torch.float16)
    ty = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}.get(kind, dt)

    def operand(rows):
        v = (torch.randint(0, 2, (rows, k), generator=q, device="cuda").float() * 2 - 1)
        buf = torch.full((rows, -(-k // 16) * 16 + 16), 99.0, device="cuda").to(ty)
        buf[:, :k] = v.to(ty)
        return buf[:, :k]

    a, w = operand(m), operand(n)
    res = torch.randint(-8, 9, (m, n), generator=q, device="cuda").to(dt)
    v = mm(a.double(), w.double().t())
    out, p = g.linear(a, w.t(), None, res, activation="relu", out_dtype=dt, pack_pre=True)
    assert torch.equal(out, (v.clamp(min=0) + res.double()).float().to(dt))
    assert torch.equal(g.linear(a, w.t(), None, res, activation="relu", out_dtype=dt), out)
    want = g.pack8(v.to(dt)) if k <= 256 else None   # whole numbers that dt holds
    if want is not None:
        assert torch.equal(p.values, want.values)
        assert torch.equal(p.scale.float(), want.scale.float())
    else:
        back = p.values.double() * p.scale.float().double().repeat_interleave(32, 1)[:, :n]
        step = p.scale.float().double().repeat_interleave(32, 1)[:, :n]
        assert bool(((back - v).abs() <= step).all())


def test_result_in_the_residuals_memory():
    q = gen(9)
    for m, n, k in ((100, 5, 64), (300, 257, 64)):
        a, b = normal(q, (m, k), torch.float16), normal(q, (n, k), torch.float16).t()
        res = normal(q, (m, n), torch.float16)
        want = g.linear(a, b, residual=res)
        got = g.linear(a, b, residual=res, out=res)
        assert got is res and torch.equal(got, want)
