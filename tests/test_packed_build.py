"""The wait states of the large tile's other asm-MFMA kernels in the built library (CPU only)."""
import os

import pytest

from dense_gemm_f16f32_amd import build as b

needs_library = pytest.mark.skipif(not os.path.exists(b.LN_SO), reason="library not built")


@needs_library
def test_wait_states_around_the_other_asm_mfmas():
    """int8; packing in four storage orders of two 16-bit types, in e4m3 and int8; column sums in two
    orders of two types."""
    assert b.check_mfma_waits(b.LN_SO, b.ASM_MORE_MFMA_KERNELS) == 15


def test_the_scan_finds_an_early_read_in_them():
    asm = "\n".join(["", "0000000000001000 <_ZN2lk13lin_more_ringILi8E>:",
                     "\tv_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], a[0:3]  // 0",
                     "\tv_accvgpr_read_b32 v0, a0  // 4"])
    assert b.scan_mfma_waits(asm, b.ASM_MORE_MFMA_KERNELS)[1]
    drained = asm.replace("\tv_accvgpr_read", "\ts_nop 7\n" * 4 + "\tv_accvgpr_read")
    assert b.scan_mfma_waits(drained, b.ASM_MORE_MFMA_KERNELS) == (1, [])
    assert b.scan_mfma_waits(asm) == (0, [])
