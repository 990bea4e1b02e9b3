"""Operands that are no tensors, on a given stream: the same TypeError as without one."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402

pytestmark = pytest.mark.gpu


def ones(*shape, dtype=torch.float16):
    return torch.ones(shape, device="cuda").to(dtype)


def test_operands_that_are_no_tensors_on_a_given_stream():
    s = torch.cuda.Stream()
    for call in (lambda: g.linear(None, ones(8, 16), stream=s), lambda: g.rms_norm(3, ones(8), stream=s),
                 lambda: g.linear_backward(None, ones(4, 8), ones(8, 16), stream=s),
                 lambda: g.rms_norm_backward(None, ones(4, 8), ones(8), ones(4), stream=s)):
        with pytest.raises(TypeError):
            call()
