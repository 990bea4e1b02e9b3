"""Products of few rows with more columns than one launch has threads for in the narrowest
workgroups.  Up to 12 GB of GPU memory."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402

pytestmark = pytest.mark.gpu

F16 = torch.float16


@pytest.mark.parametrize("n", [2 ** 27 + 16, 2 ** 29 + 8])
def test_products_of_many_columns(n):
    """More columns than a launch has threads for in workgroups of 16, and of 64."""
    print(f"linear 2 x {n} x 8", flush=True)
    a = torch.zeros((2, 8), dtype=F16, device="cuda")
    a[0, 0], a[1, 7] = 1, 2
    b = torch.zeros((n, 8), dtype=F16, device="cuda")
    b[0], b[n // 2, 7], b[n - 1] = 1, 3, 5
    got = g.linear(a, b.t())
    places = [0, 1, n // 2, n - 2, n - 1]
    assert got[0, places].tolist() == [1, 0, 0, 0, 5]
    assert got[1, places].tolist() == [2, 0, 6, 0, 10]
    assert int(got.count_nonzero()) == 5
