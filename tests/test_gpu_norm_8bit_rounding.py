"""The 8-bit norm's values are the quotients y / scale, rounded once to fp32 and once to e4m3.

With the norm's own rstd and scale, the plain quotient is made of the same fp32 operations (h, h
rstd, times weight, over scale, each rounded once), so the values have to be equal: a quotient
taken as a product with the rounded 1 / scale is off by up to 2^-23 of itself, and lands on the
other side of a tie about once in 2^20 values (ties lie 2^-3 apart)."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import normal  # noqa: E402

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def plain_values(x, r, w, rstd, scale):
    y = (x.float() + r.float()) * rstd[:, None] * w.float()
    return (y / scale[:, None]).to(E4M3).float()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,dim", [(30000, 500), (8192, 2000), (4096, 4096), (1000, 20000)])
def test_values_are_the_rounded_quotients(rows, dim, dtype):
    q = torch.Generator(device="cuda")
    q.manual_seed(dim)
    x, r = normal(q, (rows, dim), dtype, 0.3), normal(q, (rows, dim), dtype)
    w = normal(q, (dim,), dtype, 0.2) + 1
    got = g.rms_norm(x, w, r, out_dtype=E4M3, with_rstd=True)
    assert torch.equal(got.y.float(), plain_values(x, r, w, got.rstd, got.scale))


def test_an_infinite_weight_keeps_its_quotients():
    """A column of infinities makes the scale infinite: infinity / infinity is NaN, what is
    finite over infinity 0."""
    x = torch.ones((3, 40), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(40, dtype=torch.bfloat16, device="cuda")
    w[7] = float("inf")
    got = g.rms_norm(x, w, out_dtype=E4M3)
    assert bool(got.scale.isinf().all())
    y = got.y.float()
    assert bool(y[:, 7].isnan().all())
    y[:, 7] = 0
    assert not y.any()
