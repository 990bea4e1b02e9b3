"""Checkpoints of empty matrices, which have no address, in the backward pass's argument checks (CPU
only: every call here is refused, only sized, or has nothing to launch)."""
import os

import pytest

pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from dense_gemm_f16f32_amd import linear_norm as ln  # noqa: E402
from test_packed_host import G, backward, packed  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(ln.LIB_PATH), reason="library not built")

EMPTY = packed(0, 128, scale=0)


@pytest.mark.parametrize("a_activation", range(5))
@pytest.mark.parametrize("change", [dict(m=0), dict(k=0), dict(m=0, k=0)])
def test_an_empty_a_with_any_activation(change, a_activation):
    size = backward(a=EMPTY, a_activation=a_activation, call="linear_backward_packed_workspace",
                    **change)
    assert size >= 0
    assert backward(a=EMPTY, a_activation=a_activation, da=0, db=0, dbias=0, activation=0,
                    **change) == g.OK


def test_without_columns_an_a_of_its_own_still_counts():
    assert backward(a=packed(2 * G, 128), a_activation=4, call="linear_backward_packed_workspace",
                    n=0) >= 0
    for change in (dict(), dict(n=0)):
        assert backward(a_activation=4, **change) == g.ERR_OPTS
