"""Results of at most 16 columns of a deep k, few rows and many: on tiles in slices of k, or as a pass
over a.  Operands of 1 and -1: whole numbers up to 2^24, bit for bit (e4m3, whose matrix instruction
rounds inside: within 2^-13 of the products' magnitudes)."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import half_step, mm  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8,
         "e4m3": torch.float8_e4m3fn}


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k", [(17, 1, 65536), (32, 16, 16384), (64, 8, 16399), (100, 5, 8192),
                                   (512, 9, 20000), (4096, 8, 4100), (2100, 16, 3000), (64, 16, 4096)])
def test_whole_numbers(m, n, k, kind):
    q = torch.Generator(device="cuda")
    q.manual_seed(m + n + k)
    ty = TYPES[kind]
    dt = ty if ty.itemsize == 2 else torch.bfloat16

    def operand(rows):
        buf = torch.full((rows, -(-k // 16) * 16 + 16), 99.0, device="cuda").to(ty)
        buf[:, :k] = (torch.randint(0, 2, (rows, k), generator=q, device="cuda") * 2 - 1).to(ty)
        return buf[:, :k]

    a, w = operand(m), operand(n)
    bias = torch.randint(-8, 9, (n,), generator=q, device="cuda").to(dt)
    print(f"narrow {m}x{n}x{k} {kind}", flush=True)
    buf = torch.full((m, n + 3), 7.0, dtype=dt, device="cuda")
    g.linear(a, w.t(), bias, out_dtype=dt, out=buf[:, :n])
    v = mm(a.double(), w.double().t()) + bias.double()
    got = buf[:, :n].double()
    if kind == "e4m3":
        assert bool(((got - v).abs() <= 2.0 ** -13 * k + half_step(dt) * (v.abs() + 8)).all())
    else:
        assert torch.equal(got, v.float().to(dt).double())
    assert bool((buf[:, n:] == 7.0).all())


@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("a_off,b_off,pad", [(1, 0, 0), (0, 1, 0), (1, 1, 0), (1, 0, 1), (0, 0, 1), (0, 0, 2)])
@pytest.mark.parametrize("m,n,k", [(17, 1, 64), (300, 7, 512), (4096, 1, 4096), (16384, 1, 1024),
                                   (2000, 16, 1000), (513, 260, 96)])
def test_any_address(m, n, k, a_off, b_off, pad, ty):
    """Rows at any 2-byte address, by the matrix's first one or by its stride."""
    q = torch.Generator(device="cuda")
    q.manual_seed(m + n + k)

    def operand(rows, off):
        buf = torch.full((off + rows * (k + pad) + 8,), float("nan"), device="cuda").to(TYPES[ty])
        v = torch.as_strided(buf, (rows, k), (k + pad, 1), off)
        v.copy_((torch.randint(0, 2, (rows, k), generator=q, device="cuda") * 2 - 1).to(TYPES[ty]))
        return v

    a, w = operand(m, a_off), operand(n, b_off)
    print(f"narrow {m}x{n}x{k} {ty} {a_off} {b_off} {pad}", flush=True)
    out = g.linear(a, w.t())
    assert torch.equal(out, mm(a.double(), w.double().t()).float().to(TYPES[ty]))
