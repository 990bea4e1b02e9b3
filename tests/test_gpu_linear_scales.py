"""The 8-bit layer's scales are applied one after the other: what a b scale_a scale_b needs has to
be representable, the product of the two scales need not be."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from linear_norm_util import F32, assert_close, e4m3_rows, linear64  # noqa: E402

pytestmark = pytest.mark.gpu


# few rows; a tile that the matrix cuts, one that it fills, 128 x 128 and 256 x 256 tiles, k slices
@pytest.mark.parametrize("m,n,k", [(1, 64, 256), (16, 100, 8192), (65, 70, 128), (64, 64, 256),
                                   (40, 70, 8192), (2048, 2048, 256), (3584, 3840, 640)])
def test_scales_whose_product_is_subnormal(m, n, k):
    """scale_a as the norm gives it for a tiny row (2^-126); the results are around 2^-120."""
    q = torch.Generator(device="cuda")
    q.manual_seed(k)
    a, _ = e4m3_rows(torch.randn((m, k), generator=q, device="cuda"))
    w, sb = e4m3_rows(torch.randn((n, k), generator=q, device="cuda") * 2.0 ** -12)
    sa = torch.full((m,), 2.0 ** -126, device="cuda")
    got = g.linear(a, w.t(), scale_a=sa, scale_b=sb)
    want, _, err, _ = linear64(a, w.t(), scale_a=sa, scale_b=sb)
    assert float(want.abs().max()) > 2.0 ** -126
    # two products with the scales; fp32's smallest step where they end below 2^-126
    assert_close(got, want, err + 4 * F32 * want.abs() + 2.0 ** -148, f"{m}x{n}x{k}")


def test_scales_whose_product_overflows():
    for m in (2, 64):
        a = torch.zeros((m, 128), device="cuda").to(torch.float8_e4m3fn)
        w = torch.ones((64, 128), device="cuda").to(torch.float8_e4m3fn)
        big = torch.full((64,), 1e25, device="cuda")
        got = g.linear(a, w.t(), scale_a=big[:m], scale_b=big)
        assert not got.any()
