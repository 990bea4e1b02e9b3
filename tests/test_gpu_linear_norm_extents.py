"""Extents up to 2^31 - 1, where an index one step past the end does not fit 31 bits: sparse whole
numbers with values at both ends, whose results are exact.  Up to 40 GB of GPU memory."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1
F16 = torch.float16


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of free GPU memory")
    yield
    torch.cuda.empty_cache()


def constant(value, *shape, dtype=F16):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.fill_(value)


def line(values, dtype=F16):
    """A row of TOP zeros with values at the given places, and a NaN right after it."""
    t = torch.zeros(TOP + 1, dtype=dtype, device="cuda")
    t[-1] = float("nan")
    for at, v in values.items():
        t[at] = v
    return t[:TOP][None, :]


def all_equal(t, value):
    """Without a temporary of t's size in a wider type."""
    return all(bool((c == value).all()) for c in t.reshape(-1).split(1 << 28))


def test_norm_of_one_row():
    print("norm 1 x 2^31 - 1", flush=True)
    x, w = constant(1, 1, TOP), constant(1, TOP)
    x[0, -1] = 3
    got = g.rms_norm(x, w, eps=0.0, with_rstd=True)
    # the mean square is 1 + 2^-28
    assert abs(got.rstd.item() - 1) <= 2.0 ** -22
    assert all_equal(got.y[0, :-1], 1) and got.y[0, -1].item() == 3


def test_8_bit_norm_of_one_row():
    print("8-bit norm 1 x 2^31 - 1", flush=True)
    x, w = constant(1, 1, TOP), constant(1, TOP)
    x[0, -1] = 2
    got = g.rms_norm(x, w, eps=0.0, out_dtype=torch.float8_e4m3fn)
    assert abs(got.scale.item() * 224 - 1) <= 2.0 ** -21
    # e4m3 of 224 and 448, as bytes
    y = got.y.view(torch.uint8)
    assert all_equal(y[0, :-1], 0x76) and y[0, -1].item() == 0x7E


def test_norm_backward_of_one_row():
    """g = x^ = 1 but for dy's last value: dx = 1 - mean + dh, dweight = dy."""
    print("norm backward 1 x 2^31 - 1", flush=True)
    dy, h, w, dh = (constant(v, *s) for v, s in ((1, (1, TOP)), (1, (1, TOP)), (1, (TOP,)),
                                                 (2, (1, TOP))))
    dy[0, -1] = 0
    dx, dw = g.rms_norm_backward(dy, h, w, torch.ones(1, device="cuda"), dh=dh)
    assert all_equal(dx[0, :-1], 2) and dx[0, -1].item() == 1
    assert all_equal(dw[:-1], 1) and dw[-1].item() == 0


@pytest.mark.parametrize("dtype", [F16, torch.bfloat16])
def test_one_deep_product(dtype):
    print("linear 1 x 1 x 2^31 - 1", flush=True)
    a = line({0: 1, 2 ** 30: 2, TOP - 1: 3}, dtype)
    b = line({0: 1, 2 ** 30 + 1: 7, TOP - 2: 9, TOP - 1: 5}, dtype)
    assert g.linear(a, b.t()).item() == 16


def test_one_deep_8_bit_product():
    print("8-bit linear 1 x 1 x 2^31 - 1", flush=True)
    one, three, five, nan = 0x38, 0x44, 0x4A, 0x7F   # in e4m3

    def bytes8(last):
        t = torch.zeros((1, TOP + 1), dtype=torch.uint8, device="cuda")
        t[0, 0], t[0, TOP - 1], t[0, TOP] = one, last, nan
        return t.view(torch.float8_e4m3fn)

    a, b = bytes8(three), bytes8(five)
    assert g.linear(a[:, :TOP], b[:, :TOP].t(), out_dtype=F16).item() == 16


def test_deep_product_of_a_row_major_b():
    print("linear 1 x 4 x 2^31 - 1", flush=True)
    a = line({0: 1, TOP - 1: 3})
    b = torch.zeros((TOP + 1, 4), dtype=F16, device="cuda")
    b[0], b[TOP - 1], b[TOP] = 1, torch.arange(4, device="cuda").half(), float("nan")
    assert g.linear(a, b[:TOP])[0].tolist() == [1, 4, 7, 10]


def test_bias_gradient_of_many_rows():
    print("bias gradient 2^31 - 1 x 8", flush=True)
    dc = torch.zeros((TOP, 8), dtype=F16, device="cuda")
    dc[0, 0], dc[TOP // 2, 1], dc[TOP - 1, 3] = 1, 2, 3
    a, b = torch.empty((TOP, 0), dtype=F16, device="cuda"), torch.empty((0, 8), dtype=F16, device="cuda")
    dbias = g.linear_backward(dc, a, b, bias_grad=True, a_grad=False, b_grad=False)[2]
    assert dbias.tolist() == [1, 2, 0, 3, 0, 0, 0, 0]


def test_products_of_many_rows():
    """The last tile's corner plus a tile's height is 2^31."""
    print("linear 2^31 - 1 x 5 x 3", flush=True)
    a = torch.zeros((TOP, 3), dtype=F16, device="cuda")
    a[0], a[TOP - 1] = 1, 2
    b = torch.ones((3, 5), dtype=F16, device="cuda")
    got = g.linear(a, b)
    assert bool((got[0] == 3).all()) and bool((got[TOP - 1] == 6).all())
    assert not got[1:1000].any() and not got[-1000:-1].any()
