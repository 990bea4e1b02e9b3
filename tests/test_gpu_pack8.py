"""Activations kept in 8 bits (pack8, unpack8, linear's pack_pre) and the backward pass that reads
them, on the GPU.  Scales are powers of two, so packing and restoring have one answer each, and
results are compared bit for bit; products as in linear_norm_util.py."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import (F32, act, assert_close, half_step, mm, normal, slope,  # noqa: E402
                              strided)

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
LOWEST = {torch.float16: -24, torch.bfloat16: -120}


def gen(seed):
    q = torch.Generator(device="cuda")
    q.manual_seed(seed)
    return q


def packed64(v, dt):
    """(integers, exponents of the scales) of finite v in 64 bits, a block of 32 columns at a
    time."""
    whole, exps = torch.empty_like(v), []
    for c in range(0, v.shape[1], 32):
        x = v[:, c:c + 32]
        top = x.abs().amax(1)
        e = torch.where(top > 0, torch.frexp(top).exponent - 7, LOWEST[dt])
        e = e.clamp(min=LOWEST[dt]).double()
        whole[:, c:c + 32] = torch.round(x / torch.exp2(e)[:, None]).clamp(-127, 127)
        exps.append(e)
    return whole, torch.stack(exps, 1)


def restored(p):
    s = p.scale.float().double().repeat_interleave(32, 1)[:, :p.values.shape[1]]
    return p.values.double() * s


def odd_packed(q, rows, dim, dt, pad=3):
    """A packed matrix whose values and scales have strides and alignments of their own."""
    p = g.pack8(normal(q, (rows, dim), dt, 2.0))
    blocks = p.scale.shape[1]
    v = torch.full((rows * (dim + pad) + 9,), 99, dtype=torch.int8, device="cuda")
    v = torch.as_strided(v, (rows, dim), (dim + pad, 1), pad)
    s = torch.full((rows * (blocks + pad) + 9,), 255, dtype=torch.uint8, device="cuda")
    s = torch.as_strided(s, (rows, blocks), (blocks + pad, 1), 1)
    v.copy_(p.values)
    s.copy_(p.scale.view(torch.uint8))
    return g.Packed8(v, s.view(torch.float8_e8m0fnu))


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (2, 8), (5, 31), (5, 32), (70, 33), (17, 63),
                                      (100, 100), (33, 512), (9, 513), (300, 1000), (1, 8190),
                                      (129, 4097), (2, 33001), (5000, 40)])
def test_pack(rows, dim, ty):
    q, dt = gen(rows + dim), DT[ty]
    x = normal(q, (rows, dim), torch.float32) * torch.exp2(
        torch.randint(-30, 12, (rows, 1), generator=q, device="cuda").float())
    x = strided(x.to(dt), dim % 3, dim % 2)
    print(f"pack {rows}x{dim} {ty}", flush=True)
    p = g.pack8(x)
    whole, exps = packed64(x.double(), dt)
    assert p.values.dtype == torch.int8 and p.values.shape == x.shape
    assert p.scale.dtype == torch.float8_e8m0fnu and p.scale.shape == (rows, -(-dim // 32))
    assert torch.equal(p.values.double(), whole)
    assert torch.equal(p.scale.float().double(), torch.exp2(exps))
    back = g.unpack8(p, dtype=dt)
    assert back.dtype == dt and torch.equal(back.double(), restored(p))   # no rounding


def test_pack_extremes():
    """Subnormal numbers, the largest ones, ties, zeros, infinities and NaN."""
    for dt in DT.values():
        info = torch.finfo(dt)
        x = torch.zeros((8, 70), dtype=dt, device="cuda")
        x[0, :40] = info.max
        x[0, 40:] = -info.max
        x[1, 3] = info.smallest_normal
        x[1, 40] = info.smallest_normal * info.eps   # the smallest number
        x[2] = torch.arange(70, device="cuda").to(dt) + 0.5       # ties below 64 scales
        x[2, ::32] = 64.0
        x[3, 5], x[3, 40] = float("inf"), 1.0
        x[4, 33], x[4, 1] = float("nan"), 1.0
        x[5, 69] = 3.0
        x[6] = -127.75
        p = g.pack8(x)
        finite = [0, 1, 2, 5, 6, 7]
        whole, exps = packed64(x[finite].double(), dt)
        assert torch.equal(p.values[finite].double(), whole)
        assert torch.equal(p.scale[finite].float().double(), torch.exp2(exps))
        back = g.unpack8(p, dtype=dt)
        assert torch.equal(back[finite].double(), restored(g.Packed8(p.values[finite],
                                                                     p.scale[finite])))
        # a block with an infinity or a NaN is NaN, its neighbours are not
        assert bool(back[3, :32].isnan().all()) and back[3, 40] == 1 and not back[3, 64:].any()
        assert bool(back[4, 32:64].isnan().all()) and back[4, 1] == 1


@pytest.mark.parametrize("activation", ACTS)
def test_unpack_with_an_activation(activation):
    q = gen(4)
    for dt in DT.values():
        p = odd_packed(q, 37, 203, dt)
        got = g.unpack8(p, dtype=dt, activation=activation)
        v = restored(p)
        assert_close(got, act(v, activation), 2.0 ** -20 * v.abs() + 2.0 ** -40, activation)


def whole(q, shape, top):
    return torch.randint(-top, top + 1, shape, generator=q, device="cuda").float()


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("bo", "rc")
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 33, 70), (5, 31, 64), (16, 100, 300), (3, 40, 8000), (16, 8200, 130),  # few rows
    (17, 33, 40), (64, 64, 64), (100, 257, 90), (40, 70, 5000), (130, 31, 200),           # 64 x 64
    (1900, 2050, 200), (1100, 1000, 2049),                                               # 128 x 128
    (3601, 3650, 64), (4097, 4100, 130), (1500, 1500, 4096)])                            # 256 x 256
def test_linear_packs_what_stands_before_the_activation(m, n, k, bo, ty):
    """Operands of 1 and -1: the value before the activation is a whole number, exact in fp32."""
    q, dt = gen(m + n + k), DT[ty]
    a = strided((whole(q, (m, k), 1) * 2 - 1).clamp(min=-1).to(dt), k % 2)
    b = (whole(q, (k, n), 1) * 2 - 1).clamp(min=-1).to(dt)
    b = strided(b if bo == "r" else b.t().contiguous().t(), k % 3)
    bias = (whole(q, (n,), 8) * 0.25).to(dt)
    res = normal(q, (m, n), dt)
    print(f"linear packing {m}x{n}x{k} {ty} {bo}", flush=True)
    out, p = g.linear(a, b, bias, res, activation="silu", pack_pre=True)
    assert torch.equal(out, g.linear(a, b, bias, res, activation="silu", with_pre=True)[0]) or m <= 16
    v = mm(a.double(), b.double()) + bias.double()
    want, exps = packed64(v, dt)
    assert isinstance(p, g.Packed8) and p.values.shape == (m, n)
    assert torch.equal(p.values.double(), want)
    assert torch.equal(p.scale.float().double(), torch.exp2(exps))
    assert_close(out, act(v, "silu") + res.double(), 2.0 ** -20 * v.abs() + 2 * F32 * (
        v.abs() + res.double().abs()))


@pytest.mark.parametrize("kind", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("m,n,k", [(1, 40, 64), (9, 33, 5000), (100, 90, 200), (1900, 2050, 530)])
def test_linear_packs_on_8_bit_operands(m, n, k, kind):
    q = gen(m + n)
    pad = -(-k // 16) * 16

    def rows8(x):
        buf = torch.zeros((x, pad), device="cuda").to(kind)
        buf[:, :k] = ((whole(q, (x, k), 1) * 2 - 1).clamp(min=-1)).to(kind)
        return buf[:, :k]

    a, w = rows8(m), rows8(n)
    out, p = g.linear(a, w.t(), activation="relu", out_dtype=torch.float16, pack_pre=True)
    v = mm(a.double(), w.double().t())
    want, exps = packed64(v, torch.float16)
    assert torch.equal(p.values.double(), want)
    assert torch.equal(p.scale.float().double(), torch.exp2(exps))
    assert torch.equal(out, v.clamp(min=0).half())


def test_linear_keeps_what_lies_around_its_checkpoint():
    """Nothing is written past a row's end, for row lengths that leave part of a block."""
    for m, n in ((3, 45), (70, 77), (300, 300)):
        a = torch.ones((m, 16), dtype=torch.float16, device="cuda")
        out, p = g.linear(a, a[:1].expand(n, 16).t().contiguous(), pack_pre=True)
        assert bool((p.values == 64).all()) and bool((p.scale.float() == 0.25).all())
        assert bool((out == 16).all())


def check_backward(m, n, k, ty, bo="c", activation="none", a_activation="none", keep="both", seed=1):
    dt = DT[ty]
    q = gen(seed)
    b = normal(q, (k, n) if bo == "r" else (n, k), dt, k ** -0.5)
    b = strided(b if bo == "r" else b.t(), m % 3, m % 2)
    dc = strided(normal(q, (m, n), dt), n % 3)
    a8, pre8 = odd_packed(q, m, k, dt), odd_packed(q, m, n, dt)
    if keep == "pre":
        a8 = g.unpack8(a8, dtype=dt)
    a64 = restored(a8) if keep != "pre" else a8.double()
    pre = pre8 if keep != "a" else g.unpack8(pre8, dtype=dt)
    what = f"backward {m}x{n}x{k} {ty} {bo} {activation} {a_activation} {keep}"
    print(what, flush=True)
    da, db, dbias = g.linear_backward(dc, a8, b, pre if activation != "none" else None,
                                      activation=activation, a_activation=a_activation,
                                      bias_grad=True)
    d, derr = dc.double(), 0.0 * dc.double()
    rerr = derr
    if activation != "none":
        p64 = restored(pre8)
        d = d * slope(p64, activation)
        derr = 2.0 ** -20 * (1 + p64.abs()) * dc.double().abs()
        rerr = derr + half_step(dt) * d.abs() + 2.0 ** -25   # rounded before the products
    aerr = 0.0 * a64
    if a_activation != "none":
        a64 = act(a64, a_activation)
        aerr = half_step(dt) * a64.abs() + 2.0 ** -19 * restored(a8).abs() + 2.0 ** -25
    b64, mag, amag = b.double(), d.abs() + rerr, a64.abs() + aerr
    assert_close(da, mm(d, b64.t()),
                 mm(rerr, b64.abs().t()) + (n + 8) * F32 * mm(mag, b64.abs().t()), what + " da")
    assert_close(db, mm(a64.t(), d), mm(a64.abs().t(), rerr) + mm(aerr.t(), mag)
                 + (m + 8) * F32 * mm(amag.t(), mag), what + " db")
    assert_close(dbias, d.sum(0), derr.sum(0) + (m + 8) * F32 * mag.sum(0), what + " dbias")
    if keep == "both":
        got = g.linear_backward(dc, a8, b, pre if activation != "none" else None,
                                activation=activation, a_activation=a_activation, a_grad=False)
        assert got[0] is None and got[2] is None and got[1].shape == (k, n)
        got = g.linear_backward(dc, a8, b, pre if activation != "none" else None,
                                activation=activation, a_activation=a_activation, b_grad=False)
        assert got[1] is None and got[0].shape == (m, k)


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("bo", "rc")
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 70, 33), (5, 64, 64), (70, 17, 129),
                                   (130, 200, 90), (513, 1025, 31), (4, 7, 5)])
def test_backward(m, n, k, bo, ty):
    check_backward(m, n, k, ty, bo, ACTS[(m + n + k) % 5], seed=m + k)
    check_backward(m, n, k, ty, bo, ACTS[(m + n) % 5], keep="a", seed=m + k)
    check_backward(m, n, k, ty, bo, ACTS[1 + (m + n) % 4], keep="pre", seed=m + k)


@pytest.mark.parametrize("activation", ACTS)
def test_backward_activations(activation):
    check_backward(100, 72, 40, "f16", "c", activation, seed=2)
    check_backward(100, 72, 40, "bf16", "r", "none", activation, seed=3)
    check_backward(100, 72, 40, "f16", "r", activation, "silu", seed=4)


@pytest.mark.parametrize("m,n,k,ty", [(2100, 1900, 200, "bf16"), (3700, 300, 3650, "f16"),
                                      (300, 3700, 3650, "bf16"), (6000, 100, 130, "f16")])
def test_backward_large(m, n, k, ty):
    check_backward(m, n, k, ty, "c", "gelu_tanh", seed=m)
    check_backward(m, n, k, ty, "r", "none", "gelu_tanh", seed=n)


def test_backward_equals_the_one_on_restored_operands():
    """Restoring rounds nothing: with the same plan the results are the same bits."""
    q = gen(6)
    for m, n, k in ((600, 700, 800), (2100, 1900, 200)):
        dt = torch.bfloat16
        a8, pre8 = g.pack8(normal(q, (m, k), dt)), g.pack8(normal(q, (m, n), dt, 2.0))
        b, dc = normal(q, (k, n), dt), normal(q, (m, n), dt)
        got = g.linear_backward(dc, a8, b, pre8, activation="gelu", bias_grad=True)
        want = g.linear_backward(dc, g.unpack8(a8), b, g.unpack8(pre8), activation="gelu",
                                 bias_grad=True)
        for u, v in zip(got, want):
            assert torch.equal(u, v)


def test_backward_empty_sizes():
    q = gen(12)
    for m, n, k in ((0, 14, 10), (6, 0, 10), (6, 14, 0)):
        dt = torch.float16
        a8, pre8 = g.pack8(normal(q, (m, k), dt)), g.pack8(normal(q, (m, n), dt))
        da, db, dbias = g.linear_backward(normal(q, (m, n), dt), a8, normal(q, (k, n), dt), pre8,
                                          activation="silu", bias_grad=True)
        assert da.shape == (m, k) and db.shape == (k, n) and dbias.shape == (n,)
        assert not da.any() if n == 0 else True
        assert not db.any() and not dbias.any() if m == 0 else True


@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu"])
def test_a_step_against_autograd(activation):
    """An MLP's two layers, forward with checkpoints and backward from them, against autograd in
    64 bits.  Norm-wise: a checkpoint's half step is at most 2^-7 of its block's largest magnitude,
    below 3 of the deviations of normal values, and uniform, hence 3 2^-7 / sqrt(3) of the norm at
    most for the value kept; it enters db of its own layer by a factor of 1 and, through the slope,
    of magnitude up to 1.13 and itself with a slope of up to 0.8, the gradients by at most 1."""
    q, dt = gen(31), torch.float16
    m, dim, hidden = 300, 200, 500
    x, dout = normal(q, (m, dim), dt), normal(q, (m, dim), dt)
    up, down = normal(q, (hidden, dim), dt, dim ** -0.5), normal(q, (dim, hidden), dt, hidden ** -0.5)
    bias = normal(q, (hidden,), dt, 0.1)
    u, pre = g.linear(x, up.t(), bias, activation=activation, pack_pre=True)
    out = g.linear(u, down.t())
    x8 = g.pack8(x)
    du, d_down, _ = g.linear_backward(dout, pre, down.t(), a_activation=activation)
    dx, d_up, d_bias = g.linear_backward(du, x8, up.t(), pre, activation=activation,
                                         bias_grad=True)
    leaves = [t.double().cpu().requires_grad_() for t in (x, up, bias, down)]
    x64, up64, bias64, down64 = leaves
    want = act(x64 @ up64.t() + bias64, activation) @ down64.t()
    want.backward(dout.double().cpu())

    def off(got, ref):
        return ((got.double().cpu() - ref).norm() / ref.norm()).item()

    assert off(out, want.detach()) <= 8 * 2.0 ** -11
    for got, leaf in zip((dx, d_up.t(), d_bias, d_down.t()), leaves):
        assert off(got, leaf.grad) <= 2 * 3 * 2.0 ** -7 / 3 ** 0.5


def test_another_stream_and_graph_replays():
    q = gen(9)
    dt = torch.bfloat16
    x, w, dc = normal(q, (70, 500), dt), normal(q, (90, 500), dt, 0.05), normal(q, (70, 90), dt)

    def step(stream=None):
        out, pre = g.linear(x, w.t(), activation="gelu", pack_pre=True, stream=stream)
        x8 = g.pack8(x, stream=stream)
        return (out, pre.values, pre.scale.view(torch.uint8), x8.values,
                g.unpack8(x8, stream=stream),
                *g.linear_backward(dc, x8, w.t(), pre, activation="gelu", bias_grad=True,
                                   stream=stream))

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
        x.copy_(normal(q, (70, 500), dt))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for u, v in zip(held, want):
            assert torch.equal(u, v)
