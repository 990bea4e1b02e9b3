"""The backward pass from a checkpoint whose block holds an infinity or a NaN: the block's 32 values are
lost, and its gradients are NaN with every activation, relu (whose slope of NaN is 0) among them."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from test_gpu_pack8 import ACTS, DT  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("activation", ACTS[1:])
@pytest.mark.parametrize("m,n,k", [(3, 70, 40), (300, 700, 64), (9, 45, 8)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_lost_block_has_no_gradients(value, m, n, k, activation, ty):
    dt = DT[ty]
    pre = torch.ones((m, n), dtype=dt, device="cuda")
    pre[1, 33] = value
    dc = torch.ones((m, n), dtype=dt, device="cuda")
    b = torch.ones((k, n), dtype=dt, device="cuda")
    da, db, dbias = g.linear_backward(dc, torch.ones((m, k), dtype=dt, device="cuda"), b, g.pack8(pre),
                                      activation=activation, bias_grad=True)
    lost = torch.zeros(n, dtype=torch.bool, device="cuda")
    lost[32:64] = True
    assert torch.equal(dbias.isnan(), lost)
    assert torch.equal(db.isnan(), lost.expand(k, n))
    rows = torch.arange(m, device="cuda") == 1
    assert torch.equal(da.isnan(), rows[:, None].expand(m, k))
