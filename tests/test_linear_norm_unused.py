"""Fields that a call says it does not read are not checked either (CPU only; made-up addresses, and
no GPU: what passes the checks fails at the launch)."""
import os

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from dense_gemm_f16f32_amd import linear_norm as ln  # noqa: E402
from test_linear_norm_host import G, backward, norm_backward  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(ln.LIB_PATH) or torch.cuda.is_available(),
                                reason="needs the library and no GPU")

LARGE = dict(m=4096, n=4096, k=4096, dc_row=4096, a_row=4096, b_col=4096, pre_row=4096, da_row=4096,
             db_col=4096)


@pytest.mark.parametrize("pre,pre_row", [(8 * G, 4096), (8 * G + 2, 1 << 50), (G, -5), (G, 0),
                                         (3, 7)])
def test_pre_without_an_activation(pre, pre_row):
    """Whatever it holds: in the workspace, of no shape, at an odd address."""
    change = dict(LARGE, activation=0, pre=pre, pre_row=pre_row)
    assert backward("linear_backward_workspace", **change) > 0
    assert backward(**change) == g.ERR_HIP


def test_pre_with_an_activation_is_still_checked():
    assert backward(**dict(LARGE, pre=8 * G)) == g.ERR_OVERLAP
    assert backward(**dict(LARGE, pre_row=-5)) == g.ERR_LD


def test_the_norms_workspace_without_a_weight_gradient():
    assert norm_backward(dweight=0, workspace=2 * G) == g.ERR_HIP
