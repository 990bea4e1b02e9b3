"""Checkpoints written through the C entry points into memory of any stride and alignment (the Python
functions' own lies on 16-byte boundaries): the same values, and not a byte beside them.  Row lengths
that leave part of a block, for every kernel that packs."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_f16f32_amd as g  # noqa: E402
from dense_gemm_f16f32_amd import linear_norm as ln  # noqa: E402
from linear_norm_util import normal, strided  # noqa: E402
from test_gpu_pack8 import DT, gen  # noqa: E402
from test_packed_host import FORWARD, PACKED, fields  # noqa: E402

pytestmark = pytest.mark.gpu

KINDS = {"f16": (torch.float16, 0), "bf16": (torch.bfloat16, 1),
         "e4m3": (torch.float8_e4m3fn, 2), "int8": (torch.int8, 8)}


class Guarded:
    """rows x cols elements of `size` bytes, `pad` more of them a row and `offset` before the first, in
    memory filled with 0x5A."""

    def __init__(self, rows, cols, size, pad, offset):
        self.size, self.row, self.cols = size, cols + pad, cols
        self.bytes = torch.full(((offset + rows * self.row + 16) * size,), 0x5A, dtype=torch.uint8,
                                device="cuda")
        self.view = torch.as_strided(self.bytes, (rows, cols * size), (self.row * size, 1),
                                     offset * size)

    def equals(self, want):
        return torch.equal(self.view, want.contiguous().view(torch.uint8))

    def untouched(self):
        b = self.bytes.clone()
        torch.as_strided(b, self.view.shape, self.view.stride(), self.view.storage_offset()).fill_(0x5A)
        return bool((b == 0x5A).all())


def packed_into(rows, dim, pad):
    values = Guarded(rows, dim, 1, pad, 1)
    scale = Guarded(rows, -(-dim // 32), 1, pad + 1, 3)
    return values, scale, fields(PACKED, dict(
        values=values.view.data_ptr(), values_row=values.row, scale=scale.view.data_ptr(),
        scale_row=scale.row), {})


def check(values, scale, want, what):
    assert values.equals(want.values), what + " values"
    assert scale.equals(want.scale.view(torch.uint8)), what + " scale"
    assert values.untouched() and scale.untouched(), what + " beside them"


@pytest.mark.parametrize("ty", DT)
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 31), (9, 33), (70, 45), (33, 512), (9, 513),
                                      (300, 1001), (129, 4097), (2, 33001)])
@pytest.mark.parametrize("pad", [0, 1, 6])
def test_pack(rows, dim, pad, ty):
    x = strided(normal(gen(dim), (rows, dim), DT[ty]), pad, pad % 2)
    values, scale, out = packed_into(rows, dim, pad)
    print(f"pack {rows}x{dim} {ty} {pad}", flush=True)
    head = fields(["rows", "dim", "type", "x", "x_row"], dict(
        rows=rows, dim=dim, type=int(ty == "bf16"), x=x.data_ptr(), x_row=dim + pad), {})
    stream = fields(["stream"], dict(stream=torch.cuda.current_stream().cuda_stream), {})
    assert ln.lib().pack8(head + out + stream) == g.OK
    check(values, scale, g.pack8(x), f"pack {rows}x{dim}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bo", "cr")
@pytest.mark.parametrize("m,n,k", [
    (1, 45, 70), (16, 100, 8), (3, 45, 8000), (16, 8200, 130),          # few rows, in slices too
    (17, 7, 600), (300, 16, 300),                                       # at most 16 columns
    (70, 77, 64), (40, 70, 5000), (130, 31, 200),                       # 64 x 64, in slices
    (1900, 2050, 200), (1100, 1001, 2049),                              # 128 x 128
    (3601, 3650, 64), (1500, 1501, 4096), (4097, 4100, 130)])           # 256 x 256, cut
def test_linear(m, n, k, bo, kind):
    ty, code = KINDS[kind]
    eight = code in (2, 8)
    if eight and bo == "r":
        return   # k-contiguous
    dt = torch.bfloat16 if eight else ty
    q = gen(m + n + k)

    def operand(rows, cols):
        v = torch.randint(-3, 4, (rows, cols), generator=q, device="cuda").float()
        pad = -(-cols // 16) * 16 - cols if eight else cols % 3
        buf = torch.zeros((rows, cols + pad), device="cuda").to(ty)
        buf[:, :cols] = v.to(ty)
        return buf[:, :cols]

    a = operand(m, k)
    b = operand(n, k).t() if bo == "c" else operand(k, n)
    bias = normal(q, (n,), dt)
    print(f"linear packing {m}x{n}x{k} {kind} {bo}", flush=True)
    want_out, want = g.linear(a, b, bias, activation="silu", out_dtype=dt, pack_pre=True)
    values, scale, pre = packed_into(m, n, 5)
    out = Guarded(m, n, 2, 3, 1)
    d = dict(m=m, n=n, k=k, type=code, out_type=int(dt == torch.bfloat16), activation=4,
             a=a.data_ptr(), a_row=a.stride(0), a_col=a.stride(1), b=b.data_ptr(),
             b_row=b.stride(0), b_col=b.stride(1), bias=bias.data_ptr(), out=out.view.data_ptr(),
             out_row=out.row)
    need = ln.lib().linear_forward_packed_workspace(fields(FORWARD, d, {}), pre)
    assert need >= 0
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    d.update(workspace=ws.data_ptr(), workspace_bytes=need,
             stream=torch.cuda.current_stream().cuda_stream)
    assert ln.lib().linear_forward_packed(fields(FORWARD, d, {}), pre) == g.OK
    check(values, scale, want, f"linear {m}x{n}x{k}")
    assert out.equals(want_out) and out.untouched() and bool((ws[need:] == 0x5A).all())
