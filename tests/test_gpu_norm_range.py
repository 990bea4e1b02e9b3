"""Rows whose squares leave fp32's range, above or below, while the norm of the row does not."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import F32, assert_close, normal  # noqa: E402

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


# one row shape each, and rows that no registers hold
@pytest.mark.parametrize("dim", [5, 500, 1000, 2000, 4096, 8000, 16000, 20001])
@pytest.mark.parametrize("size,eps", [(1e19, 1e-5), (1e25, 1e-5), (1e38, 1e-5), (1e-15, 1e-38),
                                      (1e-25, 0.0), (1e-30, 0.0)])
def test_rows_of_any_size(dim, size, eps):
    q = torch.Generator(device="cuda")
    q.manual_seed(dim)
    x = normal(q, (3, dim), torch.float32, 0.3).clamp(-1.5, 1.5)
    x = (x * size).bfloat16()
    x[1] = 1.0
    w = normal(q, (dim,), torch.bfloat16, 0.2) + 1
    got = g.rms_norm(x, w, eps=eps, with_rstd=True)
    h = x.double()
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None] * w.double()
    rel = (dim + 16) * F32
    assert bool(((got.rstd.double() - rstd).abs() <= rel * rstd).all())
    assert_close(got.y, y, rel * y.abs(), "y")
    eight = g.rms_norm(x, w, eps=eps, out_dtype=E4M3)
    scale = y.abs().amax(1) / 448
    assert bool(((eight.scale.double() - scale).abs() <= rel * scale).all())
    back = eight.y.double() * eight.scale.double()[:, None]
    assert bool(((back - y).abs() <= (2.0 ** -4 + rel) * y.abs() + 2.0 ** -10 * scale[:, None]).all())
