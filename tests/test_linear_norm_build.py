"""What the build checks in the linear layer's and the norm's library (CPU only): the wait states
of its inline-asm MFMAs, and that no kernel keeps an array in memory."""
import os

import pytest

from dense_gemm_f16f32_amd import build as b

needs_library = pytest.mark.skipif(not os.path.exists(b.LN_SO), reason="library not built")


@needs_library
def test_wait_states_around_the_asm_mfmas():
    """The 256 x 256 tile: four storage orders of two 16-bit types, one of e4m3."""
    assert b.check_mfma_waits(b.LN_SO) == 9


@needs_library
def test_no_kernel_keeps_an_array_in_memory():
    assert b.kernels_with_private_arrays(b.LN_SO) == []


def test_the_scan_reads_kernel_descriptors(monkeypatch):
    text = "".join(f"\t.amdhsa_kernel k{i}\n\t.amdhsa_private_segment_fixed_size {p}\n"
                   f"\t.amdhsa_user_sgpr_dispatch_ptr {d}\n.end_amdhsa_kernel\n"
                   for i, (p, d) in enumerate([(0, 0), (16, 0), (0, 1)]))
    monkeypatch.setattr(b, "disassemble", lambda *a: text)
    assert b.kernels_with_private_arrays("x") == ["k1", "k2"]
