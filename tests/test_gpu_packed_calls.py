"""The layer norm's, the 8-bit rows' and the checkpoints' functions as they may be called: on another
stream with temporaries, on the largest extents, with what they refuse."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from test_gpu_linear_norm_extents import TOP, all_equal, constant, memory  # noqa: E402,F401
from test_gpu_linear_norm_streams import on_another_stream, ones  # noqa: E402

pytestmark = pytest.mark.gpu

F16, BF16, I8, E4M3 = torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn


def t(*shape, dtype=F16):
    return torch.ones(shape, device="cuda").to(dtype)


def packed(rows, dim):
    return g.pack8(t(rows, dim))


def test_temporaries_of_a_call_on_another_stream():
    n = 512
    r = on_another_stream(lambda s: g.layer_norm(ones(n, n), ones(n), ones(n), ones(n, n),
                                                 with_stats=True, stream=s))
    assert bool((r.y == 1).all()) and bool((r.h == 2).all()) and bool((r.mean == 2).all())
    dx, dw, db = on_another_stream(lambda s: g.layer_norm_backward(
        ones(n, n), ones(n, n), ones(n), torch.zeros(n, device="cuda"),
        torch.ones(n, device="cuda"), dh=ones(n, n), stream=s))
    # g = x^ = 1: the mean of g and that of g x^ are 1 each
    assert bool((dx == 0).all()) and bool((dw == n).all()) and bool((db == n).all())
    q = on_another_stream(lambda s: g.quantize_rows(ones(n, n), stream=s))
    assert bool((q.values == 127).all())
    p = on_another_stream(lambda s: g.pack8(ones(n, n), stream=s))
    assert bool((p.values == 64).all()) and bool((p.scale.float() == 2.0 ** -6).all())
    y = on_another_stream(lambda s: g.unpack8(g.Packed8(ones(n, n, dtype=I8),
                                                        ones(n, n // 32).to(p.scale.dtype)), stream=s))
    assert bool((y == 1).all())
    out, pre = on_another_stream(lambda s: g.linear(ones(n, n), ones(n, n), ones(n), pack_pre=True,
                                                    stream=s))
    assert bool((out == n + 1).all()) and bool((pre.values == 64).all())   # 513 / 8, rounded

    def backward(s):
        scale = ones(n, n // 32).to(p.scale.dtype)
        return g.linear_backward(ones(n, n), g.Packed8(ones(n, n, dtype=I8), scale), ones(n, n),
                                 g.Packed8(ones(n, n, dtype=I8), scale.clone()), activation="relu",
                                 bias_grad=True, stream=s)

    da, db, dbias = on_another_stream(backward)
    assert bool((da == n).all()) and bool((db == n).all()) and bool((dbias == n).all())
    out = on_another_stream(lambda s: g.linear(ones(n, n, dtype=I8), ones(n, n, dtype=I8).t(),
                                               scale_a=torch.ones(n, device="cuda"),
                                               scale_b=torch.ones(n, device="cuda"), stream=s))
    assert bool((out == n).all())


def test_two_streams_at_once():
    """Calls on two streams share nothing."""
    q = torch.Generator(device="cuda")
    q.manual_seed(1)
    xs = [torch.randn((300, 700), generator=q, device="cuda").to(BF16) for _ in range(2)]
    ws = [torch.randn((500, 700), generator=q, device="cuda").to(BF16) for _ in range(2)]
    dcs = [torch.randn((300, 500), generator=q, device="cuda").to(BF16) for _ in range(2)]
    m = torch.zeros(300, device="cuda")

    def step(i, stream=None):
        out, pre = g.linear(xs[i], ws[i].t(), activation="silu", pack_pre=True, stream=stream)
        grads = g.linear_backward(dcs[i], g.pack8(xs[i], stream=stream), ws[i].t(), pre,
                                  activation="silu", bias_grad=True, stream=stream)
        back = g.layer_norm_backward(xs[i], xs[i], ws[i][0], m, m + 1, stream=stream)
        return (out, *grads, *back)

    want = [step(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(step(i, streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for results in got[i]:
            for u, v in zip(results, want[i]):
                assert torch.equal(u, v)


@pytest.mark.parametrize("call", [
    lambda: g.layer_norm(t(4, 8), t(7)), lambda: g.layer_norm(t(4, 8), t(8), t(7)),
    lambda: g.layer_norm(t(4, 8), t(8, dtype=torch.float32)),
    lambda: g.layer_norm(t(4, 8), t(8), t(8, dtype=BF16)), lambda: g.layer_norm(t(8), t(8)),
    lambda: g.layer_norm(t(4, 8), t(8), None, t(3, 8)),
    lambda: g.layer_norm(t(4, 8), t(8), out_dtype=BF16),
    lambda: g.layer_norm(t(4, 16)[:, ::2], t(8)), lambda: g.layer_norm(t(4, 8), t(8).cpu()),
    lambda: g.layer_norm_backward(t(4, 8), t(4, 8), t(8), t(4), torch.ones(4, device="cuda")),
    lambda: g.layer_norm_backward(t(4, 8), t(4, 8), t(8), torch.ones(5, device="cuda"),
                                  torch.ones(4, device="cuda")),
    lambda: g.quantize_rows(t(8)), lambda: g.quantize_rows(t(4, 8, dtype=torch.float32)),
    lambda: g.quantize_rows(t(4, 8), dtype=F16), lambda: g.quantize_rows(t(16, 4).t()),
    lambda: g.pack8(t(8)), lambda: g.pack8(t(4, 8, dtype=I8)), lambda: g.pack8(t(16, 4).t()),
    lambda: g.unpack8(packed(4, 8), dtype=torch.float32),
    lambda: g.unpack8(packed(4, 8), activation="swish"),
    lambda: g.unpack8(g.Packed8(t(4, 8), packed(4, 8).scale)),
    lambda: g.unpack8(g.Packed8(packed(4, 64).values, packed(4, 8).scale)),
    lambda: g.unpack8(g.Packed8(packed(4, 8).values, packed(4, 8).scale.view(torch.uint8))),
    lambda: g.unpack8(g.Packed8(packed(4, 8).values, packed(4, 8).scale.cpu())),
    lambda: g.linear(t(4, 8), t(8, 16), with_pre=True, pack_pre=True),
    lambda: g.linear(t(4, 16, dtype=I8), t(8, 16, dtype=E4M3).t()),
    lambda: g.linear(t(4, 16, dtype=I8), t(8, 16, dtype=I8).t(), out_dtype=I8),
    lambda: g.linear(t(4, 16, dtype=torch.uint8), t(8, 16, dtype=torch.uint8).t()),
    lambda: g.linear_backward(t(4, 16), packed(4, 9), t(8, 16)),
    lambda: g.linear_backward(t(4, 16), packed(5, 8), t(8, 16)),
    lambda: g.linear_backward(t(4, 16), t(4, 8), t(8, 16), a_activation="silu"),
    lambda: g.linear_backward(t(4, 16), packed(4, 8), t(8, 16), activation="silu"),
    lambda: g.linear_backward(t(4, 16), packed(4, 8), t(8, 16), packed(4, 17), activation="silu"),
    lambda: g.linear_backward(t(4, 16), packed(4, 8), t(8, 16), a_activation="swish"),
])
def test_value_errors(call):
    with pytest.raises(ValueError):
        call()


def test_library_codes():
    for call, code in (
            (lambda: g.layer_norm(t(4, 0), t(0)), g.ERR_DIM),
            (lambda: g.layer_norm(t(4, 8), t(8), eps=-1.0), g.ERR_OPTS),
            (lambda: g.quantize_rows(t(4, 0)), g.ERR_DIM),
            (lambda: g.linear(t(4, 24, dtype=I8), t(24, 32, dtype=I8)), g.ERR_LD),
            (lambda: g.linear(t(4, 20, dtype=I8), t(32, 32, dtype=I8)[:, :20].t()), g.ERR_LD),
            (lambda: g.pack8(t(1, 16).expand(4, 16)), g.ERR_LD)):
        with pytest.raises(g.GemmError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("call", [
    lambda x: g.layer_norm(x, t(8)), lambda x: g.layer_norm(t(4, 8), t(8), None, x),
    lambda x: g.layer_norm_backward(t(4, 8), x, t(8), torch.ones(4, device="cuda"),
                                    torch.ones(4, device="cuda")),
    lambda x: g.quantize_rows(x), lambda x: g.pack8(x),
    lambda x: g.linear(x, t(8, 16), pack_pre=True)])
def test_a_gradient_is_not_lost_in_silence(call):
    x = t(4, 8).requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        call(x)
    with torch.no_grad():
        call(x)


def test_more_rows_than_one_launch_takes():
    rows = (1 << 21) + 5
    x = torch.ones((rows, 8), dtype=F16, device="cuda")
    x[:, ::2] = -1
    x[-1] = 3 * x[-1]
    got = g.layer_norm(x, t(8), eps=0.0, with_stats=True)
    assert bool((got.y.abs() == 1).all()) and not got.mean.any()
    assert bool((got.rstd[:-1] == 1).all()) and abs(got.rstd[-1].item() * 3 - 1) <= 2.0 ** -22
    q = g.quantize_rows(x)
    assert bool((q.values.abs() == 127).all())
    assert q.scale[-1].item() == torch.tensor(3.0 / 127, dtype=torch.float64).float().item()


def test_layer_norm_of_one_row(memory):  # noqa: F811
    print("layer norm 1 x 2^31 - 1", flush=True)
    x, w = constant(1, 1, TOP), constant(1, TOP)
    x[0, ::2] = -1   # one more of them: the mean is -2^-31
    got = g.layer_norm(x, w, eps=0.0, with_stats=True)
    assert abs(got.rstd.item() - 1) <= 2.0 ** -20 and abs(got.mean.item()) <= 2.0 ** -20
    assert all_equal(got.y[0, ::2], -1) and all_equal(got.y[0, 1::2], 1)
    del got
    got = g.layer_norm(x, w, eps=0.0, out_dtype=I8)
    assert all_equal(got.y[0, ::2], -127) and all_equal(got.y[0, 1::2], 127)
    del got
    got = g.quantize_rows(x)
    assert all_equal(got.values[0, ::2], -127) and all_equal(got.values[0, 1::2], 127)


def test_layer_norm_backward_of_one_row(memory):  # noqa: F811
    """x^ = 1 everywhere and g = 1 but for dy's last value: both means are 1 (to 2^-31)."""
    print("layer norm backward 1 x 2^31 - 1", flush=True)
    dy, h, w = constant(1, 1, TOP), constant(1, 1, TOP), constant(1, TOP)
    dy[0, -1] = 0
    dx, dw, db = g.layer_norm_backward(dy, h, w, torch.zeros(1, device="cuda"),
                                       torch.ones(1, device="cuda"))
    # whole numbers: a thread's sum stays below 2^22 and the row's, 2^31 - 2, is rounded to 2^31, whose
    # mean is 1 to 2^-23
    assert all_equal(dx[0, :-1], -1) and dx[0, -1].item() == -2
    assert all_equal(dw[:-1], 1) and dw[-1].item() == 0 and torch.equal(db, dw)


def test_checkpoint_of_one_row(memory):  # noqa: F811
    print("pack 1 x 2^31 - 1", flush=True)
    x = constant(1, 1, TOP)
    x[0, -1] = -4
    p = g.pack8(x)
    # the last block holds 31 values: 64 and less in units of 2^-4
    assert all_equal(p.values[0, :-31], 64) and p.values[0, -1].item() == -64
    assert all_equal(p.values[0, -31:-1], 16) and p.scale[0, -1].float().item() == 2.0 ** -4
    assert torch.equal(g.unpack8(p, dtype=F16)[0, -100:], x[0, -100:])


def test_checkpoint_of_many_rows(memory):  # noqa: F811
    print("pack 2^31 - 1 x 3", flush=True)
    x = torch.zeros((TOP, 3), dtype=F16, device="cuda")
    x[0], x[TOP - 1] = 1, 2
    p = g.pack8(x)
    assert bool((p.values[0] == 64).all()) and bool((p.values[-1] == 64).all())
    assert not p.values[1:1000].any() and not p.values[-1000:-1].any()
    y = g.unpack8(p, dtype=F16)
    assert torch.equal(y[:10], x[:10]) and torch.equal(y[-10:], x[-10:])
