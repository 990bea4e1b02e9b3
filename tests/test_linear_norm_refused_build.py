"""A build that fails one of the checks leaves the library that is in place alone, and nothing
beside it (CPU only; a copy of the built library stands in for the compiler's output)."""
import os

import pytest

from dense_gemm_f16f32_amd import build as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LN_SO), reason="library not built")


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A folder of its own for the library, with an older one in it, and a compiler that copies."""
    hipcc = tmp_path / "hipcc"
    hipcc.write_text(f"#!/bin/sh\nwhile [ $# -gt 1 ]; do [ $1 = -o ] && cp {b.LN_SO} $2; shift; done\n")
    hipcc.chmod(0o755)
    folder = tmp_path / "lib"
    folder.mkdir()
    so = folder / "library.so"
    so.write_text("older")
    monkeypatch.setattr(b, "HIPCC", str(hipcc))
    monkeypatch.setattr(b, "LN_SO", str(so))
    return so


def test_kernels_with_private_arrays_are_not_installed(place, monkeypatch):
    monkeypatch.setattr(b, "kernels_with_private_arrays", lambda path: ["kernel"])
    with pytest.raises(RuntimeError, match="kernel"):
        b.build_linear_norm()
    assert place.read_text() == "older" and os.listdir(place.parent) == [place.name]


def test_the_scan_sees_the_new_library(place, monkeypatch):
    seen = []
    monkeypatch.setattr(b, "kernels_with_private_arrays",
                        lambda path: seen.append(os.path.getsize(path)) or [])
    b.build_linear_norm()
    assert seen == [os.path.getsize(place)] and seen[0] > 100000
    assert os.listdir(place.parent) == [place.name]


def test_a_missing_wait_is_not_installed(place, monkeypatch):
    def violated(path):
        raise RuntimeError("before the drain")
    monkeypatch.setattr(b, "check_mfma_waits", violated)
    with pytest.raises(RuntimeError, match="drain"):
        b.build_linear_norm()
    assert place.read_text() == "older" and os.listdir(place.parent) == [place.name]
