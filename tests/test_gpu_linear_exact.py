"""The linear layer and its backward pass on operands of 1 and -1 with whole-numbered bias,
residual and gradients.  Every partial sum is a whole number below 2^24, exact in fp32 in any
order, so the results are the exact ones, rounded once: equal to the definition's, bit for bit.
One value of k or one element left out moves every result that it belongs to by 1, which f16 shows
up to 2048 and bf16 up to 256, at any depth.  The operands lie among NaN."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import mm, strided  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


def gen(seed):
    q = torch.Generator(device="cuda")
    q.manual_seed(seed)
    return q


def signs(q, shape):
    return torch.randint(0, 2, shape, generator=q, device="cuda").float() * 2 - 1


def whole(q, shape, top):
    return torch.randint(-top, top + 1, shape, generator=q, device="cuda").float()


def operand(q, rows, cols, dtype, order, pad):
    t = signs(q, (rows, cols)).to(dtype)
    return strided(t if order == "r" else t.t().contiguous().t(), pad, pad % 2)


def rounded(v, dtype):
    """The whole numbers v (float64, below 2^24) in dtype, rounded once."""
    assert float(v.abs().max()) < 2 ** 24
    return v.float().to(dtype)


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("ao,bo", ["rr", "rc", "cr", "cc"])
@pytest.mark.parametrize("m,n,k", [
    (1, 40, 8000), (5, 24, 6001), (16, 64, 8192), (3, 300, 4095),      # few rows, in k slices
    (40, 70, 5000), (100, 300, 4097), (64, 64, 16384), (33, 65, 63),   # 64 x 64, in k slices
    (1900, 2050, 200), (2048, 1920, 128), (1100, 1000, 2049),          # 128 x 128
    (3841, 3583, 447), (3584, 3840, 385), (4096, 3584, 40), (1500, 1500, 4096),
    (4097, 4100, 130), (300, 8192, 1030)])                             # cut at the last whole tile
def test_forward(m, n, k, ao, bo, ty):
    q, dt = gen(m + n + k), DT[ty]
    pad = (m + k) % 3
    a, b = operand(q, m, k, dt, ao, pad), operand(q, k, n, dt, bo, pad)
    bias, res = whole(q, (n,), 8).to(dt), whole(q, (m, n), 8).to(dt)
    print(f"exact {m}x{n}x{k} {ty} {ao}{bo}", flush=True)
    out, pre = g.linear(a, b, bias, strided(res, pad), activation="relu", with_pre=True)
    v = mm(a.double(), b.double()) + bias.double()
    assert torch.equal(pre, rounded(v, dt))
    assert torch.equal(out, rounded(v.clamp(min=0) + res.double(), dt))


@pytest.mark.parametrize("out", DT)
@pytest.mark.parametrize("m,n,k", [(1, 64, 8192), (16, 100, 5001), (9, 16, 4097), (17, 64, 512),
                                   (64, 64, 8192), (70, 90, 4999), (100, 200, 513),
                                   (1900, 2050, 511), (2048, 2048, 1030), (3584, 3840, 640),
                                   (3600, 3650, 1159)])
def test_8_bit_forward(m, n, k, out):
    q, dt = gen(m + n + k), DT[out]
    pad = -k % 16 + 16

    def rows8(x):
        buf = torch.full((x, k + pad), float("nan"), device="cuda").to(E4M3)
        buf[:, :k] = signs(q, (x, k)).to(E4M3)
        return buf[:, :k]

    a, w = rows8(m), rows8(n)
    sa = 2.0 ** whole(q, (m,), 1)
    sb = torch.full((n,), 2.0, device="cuda")
    bias, res = whole(q, (n,), 8).to(dt), whole(q, (m, n), 8).to(dt)
    got = g.linear(a, w.t(), bias, res, scale_a=sa, scale_b=sb, out_dtype=dt, activation="relu")
    v = mm(a.double(), w.double().t()) * (2 * sa.double()[:, None]) + bias.double()
    assert torch.equal(got, rounded(v.clamp(min=0) + res.double(), dt))


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("activation", ["none", "relu"])
@pytest.mark.parametrize("ao,bo", ["rr", "rc", "cr", "cc"])
@pytest.mark.parametrize("m,n,k", [
    (3, 9, 200), (64, 64, 64), (65, 127, 8), (200, 250, 70), (256, 255, 256),   # one launch
    (1024, 768, 128), (513, 1025, 31), (700, 600, 500), (4000, 64, 70),         # pairs
    (6000, 100, 130), (300, 3700, 3650), (2100, 1900, 200), (5, 4096, 64),
    (1, 70, 4000), (4097, 130, 300)])
def test_backward(m, n, k, ao, bo, activation, ty):
    q, dt = gen(m + n + k), DT[ty]
    pad = (m + k) % 3
    a, b = operand(q, m, k, dt, ao, pad), operand(q, k, n, dt, bo, pad)
    dc = strided(signs(q, (m, n)).to(dt), pad)
    pre = strided(signs(q, (m, n)).to(dt), pad) if activation == "relu" else None
    print(f"exact backward {m}x{n}x{k} {ty} {ao}{bo} {activation}", flush=True)
    da, db, dbias = g.linear_backward(dc, a, b, pre, activation=activation, bias_grad=True)
    d = dc.double() if pre is None else dc.double() * (pre > 0)
    assert torch.equal(da, rounded(mm(d, b.double().t()), dt))
    assert torch.equal(db, rounded(mm(a.double().t(), d), dt))
    assert torch.equal(dbias, rounded(d.sum(0), dt))
