"""What the linear layer's and the norm's Python functions refuse, on GPU tensors: ValueError for
what only the tensors show, GemmError with the library's code for the rest; nothing is written."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def t(*shape, dtype=torch.float16):
    return torch.ones(shape, device="cuda").to(dtype)


@pytest.mark.parametrize("call", [
    lambda: g.linear(t(4, 8), t(7, 16)),                                   # inner sizes
    lambda: g.linear(t(8), t(8, 16)),                                      # not 2-D
    lambda: g.linear(t(4, 8), t(8, 16, dtype=torch.bfloat16)),             # mixed types
    lambda: g.linear(t(4, 8, dtype=torch.float32), t(8, 16, dtype=torch.float32)),
    lambda: g.linear(t(4, 8), t(8, 16).cpu()),
    lambda: g.linear(t(4, 8), t(8, 16), t(15)),                            # bias size
    lambda: g.linear(t(4, 8), t(8, 16), t(32)[::2]),                       # bias stride
    lambda: g.linear(t(4, 8), t(8, 16), t(16, dtype=torch.float32)),
    lambda: g.linear(t(4, 8), t(8, 16), None, t(4, 15)),
    lambda: g.linear(t(4, 8), t(8, 16), None, t(16, 4).t()),               # residual order
    lambda: g.linear(t(4, 8), t(8, 16), activation="swish"),
    lambda: g.linear(t(4, 8), t(8, 16), activation=None),
    lambda: g.linear(t(4, 8), t(8, 16), out_dtype=torch.bfloat16),
    lambda: g.linear(t(4, 8), t(8, 16), out=t(4, 16, dtype=torch.bfloat16)),
    lambda: g.linear(t(4, 16, dtype=E4M3), t(8, 16, dtype=E4M3).t(), out_dtype=torch.float32),
    lambda: g.linear(t(4, 16, dtype=E4M3), t(8, 16, dtype=E4M3).t(), scale_a=t(4)),
    lambda: g.linear_backward(t(4, 16), t(4, 8), t(8, 16), activation="silu"),   # no pre
    lambda: g.linear_backward(t(4, 16), t(4, 8), t(8, 15)),
    lambda: g.linear_backward(t(4, 16, dtype=E4M3), t(4, 8), t(8, 16)),
    lambda: g.rms_norm(t(4, 8), t(7)),
    lambda: g.rms_norm(t(4, 8), t(8, dtype=torch.float32)),
    lambda: g.rms_norm(t(8), t(8)),
    lambda: g.rms_norm(t(4, 8), t(8), t(3, 8)),
    lambda: g.rms_norm(t(4, 8), t(8), out_dtype=torch.bfloat16),
    lambda: g.rms_norm_backward(t(4, 8), t(4, 8), t(8), t(4)),             # rstd's type
])
def test_value_errors(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [lambda: g.linear(None, t(8, 16)), lambda: g.linear(t(4, 8), 3),
                                  lambda: g.rms_norm(t(4, 8), None),
                                  lambda: g.linear(t(4, 8), t(8, 16), out_dtype="bf16")])
def test_type_errors(call):
    with pytest.raises(TypeError):
        call()


def test_library_codes():
    a = t(16, 16)
    for call, code in (
            (lambda: g.linear(a, t(16, 16), out=a), g.ERR_OVERLAP),
            (lambda: g.linear(t(4, 8), t(8, 16), None, t(1, 16).expand(4, 16)), g.ERR_LD),
            (lambda: g.linear(t(4, 16)[:, ::2], t(8, 16)), g.ERR_LD),
            (lambda: g.linear(t(4, 16, dtype=E4M3), t(16, 32, dtype=E4M3)), g.ERR_LD),
            (lambda: g.linear(t(4, 20, dtype=E4M3), t(32, 32, dtype=E4M3)[:, :20].t()), g.ERR_LD),
            (lambda: g.linear(t(4, 8), t(8, 16), scale_a=t(4, dtype=torch.float32)), g.ERR_OPTS),
            (lambda: g.rms_norm(t(4, 0), t(0)), g.ERR_DIM),
            (lambda: g.rms_norm(t(4, 8), t(8), eps=-1.0), g.ERR_OPTS)):
        with pytest.raises(g.GemmError) as e:
            call()
        assert e.value.code == code
    assert bool((a == 1).all())


def test_a_refused_call_leaves_the_next_one_alone():
    with pytest.raises(ValueError):
        g.linear(t(4, 8), t(7, 16))
    assert bool((g.linear(t(4, 8), t(8, 16)) == 8).all())
