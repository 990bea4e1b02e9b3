"""How results of at most 16 columns are computed, by the workspace that the call asks for (CPU only): on
tiles in slices of k, which takes some, or as a pass over a in one piece, which takes none."""
import os

import pytest

pytest.importorskip("torch")

from dense_gemm_f16f32_amd import linear_norm as ln  # noqa: E402
from test_packed_host import BF16, E4M3, F16, FORWARD, G, I8, fields  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(ln.LIB_PATH), reason="library not built")


def workspace(m, n, k, ty, a_row=None, b_col=None, a=G, b=2 * G):
    ld = -(-k // 16) * 16
    return ln.lib().linear_forward_workspace(fields(FORWARD, dict(
        m=m, n=n, k=k, type=ty, out_type=BF16 if ty in (I8, E4M3) else ty, a=a, a_row=a_row or ld,
        a_col=1, b=b, b_row=1, b_col=b_col or ld, out=3 * G, out_row=n), {}))


@pytest.mark.parametrize("ty", [F16, BF16, I8, E4M3])
@pytest.mark.parametrize("m,n,k", [(17, 1, 16384), (32, 16, 16384), (64, 8, 16384), (64, 16, 65536),
                                   (17, 1, 131071), (512, 9, 65536)])
def test_few_rows_of_a_deep_k_are_split(m, n, k, ty):
    """They have too few workgroups in one piece; the 17th column does not change the tiles."""
    assert workspace(m, n, k, ty) == workspace(m, 17, k, ty) > 0


@pytest.mark.parametrize("ty", [F16, BF16, I8, E4M3])
@pytest.mark.parametrize("m,n,k", [(4095, 1, 4096), (4096, 8, 4096), (64, 4, 4096), (2000, 1, 6000)])
def test_a_pass_over_a_where_it_is_faster(m, n, k, ty):
    assert workspace(m, n, k, ty) == 0 < workspace(m, 17, k, ty)


@pytest.mark.parametrize("m,n,k", [(64, 4, 4096), (4095, 8, 4096), (2000, 1, 6000)])
def test_rows_off_4_byte_boundaries_take_the_tiles(m, n, k):
    """Their loads take the pass over a two or three times as long.  One row of b has no stride."""
    for ty in (F16, BF16):
        tiles = workspace(m, 17, k, ty)
        assert workspace(m, n, k, ty, a_row=k + 1) == tiles > 0
        assert workspace(m, n, k, ty, a_row=k + 1, b_col=k + 3) == tiles
        assert workspace(m, n, k, ty, b_col=k + 1) == (tiles if n > 1 else 0)
        assert workspace(m, n, k, ty, a_row=k + 2, b_col=k + 6) == 0


@pytest.mark.parametrize("n", [1, 5, 16, 17, 257, 300, 4097])
@pytest.mark.parametrize("m", [17, 300, 4095, 16384])
def test_the_workspace_goes_by_no_address(m, n):
    for k in (64, 513, 4096, 16384):
        for pad in (0, 1):
            want = workspace(m, n, k, BF16, a_row=k + pad)
            for a, b in ((G + 2, 2 * G), (G, 2 * G + 2), (G + 2, 2 * G + 2)):
                assert workspace(m, n, k, BF16, a_row=k + pad, a=a, b=b) == want
