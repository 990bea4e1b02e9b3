"""Arguments that cannot be read: their own errors arrive."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402

pytestmark = pytest.mark.gpu


def ones(*shape, dtype=torch.float16):
    return torch.ones(shape, device="cuda").to(dtype)


class Unreadable:
    def __bool__(self):
        raise KeyError("no truth value")


@pytest.mark.parametrize("call", [
    lambda: g.linear(ones(4, 8), ones(8, 16), with_pre=Unreadable()),
    lambda: g.linear_backward(ones(4, 16), ones(4, 8), ones(8, 16), bias_grad=Unreadable()),
    lambda: g.linear_backward(ones(4, 16), ones(4, 8), ones(8, 16), a_grad=Unreadable()),
    lambda: g.rms_norm(ones(4, 8), ones(8), with_rstd=Unreadable()),
    lambda: g.rms_norm_backward(ones(4, 8), ones(4, 8), ones(8), torch.ones(4, device="cuda"),
                                weight_grad=Unreadable())])
def test_a_flags_own_error_arrives(call):
    with pytest.raises(KeyError, match="no truth value"):
        call()
