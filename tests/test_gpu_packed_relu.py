"""The backward pass of relu from a checkpoint: its slope is 0 or 1, so what the checkpoint has to hold is
the sign.  linear's pack_pre keeps it for values far below their block's step."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from test_gpu_pack8 import ACTS, DT, packed64  # noqa: E402

pytestmark = pytest.mark.gpu

SMALL = (3.0, -3.0, 1.0, 0.0, 0.015625, -0.015625, 4.0, -5.0)   # in a block of step 8


def outliers(n, dt):
    """Small values of both signs, and 1000 in the first column of every second block (step 8)."""
    v = torch.tensor(SMALL, device="cuda").repeat(-(-n // 8))[:n].clone()
    v[::64] = 1000.0
    return v.to(dt)


def expected(v, dt):
    whole, exps = packed64(v, dt)
    return torch.where((v > 0) & (whole == 0), torch.ones_like(whole), whole), torch.exp2(exps)


@pytest.mark.parametrize("kind", ["f16", "bf16", "int8", "e4m3"])
@pytest.mark.parametrize("bo", "cr")
@pytest.mark.parametrize("m,n,k", [(1, 40, 8), (3, 200, 5000), (16, 300, 64), (16, 8200, 130),   # few rows
                                   (40, 7, 64), (300, 16, 512),                    # at most 16 columns
                                   (64, 64, 64), (40, 70, 5000), (300, 257, 128),                # 64 x 64
                                   (1900, 2050, 200), (1100, 1000, 2049),                      # 128 x 128
                                   (3601, 3650, 64), (1500, 1500, 4096)])                      # 256 x 256
def test_linear_keeps_the_sign(m, n, k, bo, kind):
    """The product is 0, so that every row is the bias, exactly."""
    eight = kind in ("int8", "e4m3")
    if eight and bo == "r":
        return   # k-contiguous
    dt = DT.get(kind, torch.bfloat16)
    ty = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}.get(kind, dt)
    pad = -(-k // 16) * 16
    a = torch.ones((m, pad), device="cuda").to(ty)[:, :k]
    b = (torch.zeros((n, pad), device="cuda").to(ty)[:, :k].t() if bo == "c"
         else torch.zeros((k, n), dtype=ty, device="cuda"))
    bias = outliers(n, dt)
    print(f"relu packing {m}x{n}x{k} {kind} {bo}", flush=True)
    out, p = g.linear(a, b, bias, activation="relu", out_dtype=dt, pack_pre=True)
    v = bias.double().expand(m, n)
    whole, scale = expected(v, dt)
    assert torch.equal(p.values.double(), whole) and torch.equal(p.scale.float().double(), scale)
    assert torch.equal(out.double(), v.clamp(min=0))
    if eight:
        return
    rows = min(m, 200)   # counts that bf16 holds
    kept = g.Packed8(p.values[:rows], p.scale[:rows])
    dbias = g.linear_backward(torch.ones((rows, n), dtype=dt, device="cuda"), a[:rows], b, kept,
                              activation="relu", bias_grad=True, a_grad=False, b_grad=False)[2]
    assert torch.equal(dbias.double(), rows * (bias.double() > 0).double())


def test_only_relu_rounds_so():
    bias = outliers(96, torch.float16)
    a = torch.zeros((5, 32), dtype=torch.float16, device="cuda")
    b = torch.zeros((32, 96), dtype=torch.float16, device="cuda")
    want = g.pack8(bias.expand(5, 96).contiguous())
    for activation in ACTS:
        p = g.linear(a, b, bias, activation=activation, pack_pre=True)[1]
        same = torch.equal(p.values, want.values)
        assert same == (activation != "relu")
        assert torch.equal(p.scale.float(), want.scale.float())
    assert bool((want.values[:, [2, 4]] == 0).all())   # 1.0 and 2^-6 beside 1000
