"""Calls on a given stream whose operands are temporaries of another: their memory stays theirs
until the call's kernels have run."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402

pytestmark = pytest.mark.gpu


def ones(*shape, dtype=torch.float16):
    return torch.ones(shape, device="cuda").to(dtype)


def on_another_stream(call):
    """The results of a call(stream) on a stream that is still busy, its inputs (made inside and
    held by nothing but the call) freed, and memory like theirs written by the current stream."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)   # about 0.1 s
    got = call(s)
    over = [torch.full((512, 512), 7.0, dtype=torch.float16, device="cuda") for _ in range(16)]
    over += [torch.full((512,), 7.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del over
    return got


def test_temporaries_of_a_call_on_another_stream():
    n = 512

    def linear(s):
        return g.linear(ones(n, n), ones(n, n), ones(n), ones(n, n), stream=s)

    def backward(s):
        return g.linear_backward(ones(n, n), ones(n, n), ones(n, n), ones(n, n), activation="relu",
                                 bias_grad=True, stream=s)

    def norm(s):
        return g.rms_norm(ones(n, n), ones(n), ones(n, n), eps=0.0, stream=s)

    def norm_backward(s):
        return g.rms_norm_backward(ones(n, n), ones(n, n), ones(n), torch.ones(n, device="cuda"),
                                   dh=ones(n, n), stream=s)

    assert bool((on_another_stream(linear) == n + 2).all())
    da, db, dbias = on_another_stream(backward)
    assert bool((da == n).all()) and bool((db == n).all()) and bool((dbias == n).all())
    r = on_another_stream(norm)
    assert bool((r.y == 1).all()) and bool((r.h == 2).all())
    dx, dw = on_another_stream(norm_backward)
    assert bool((dx == 1).all()) and bool((dw == n).all())
