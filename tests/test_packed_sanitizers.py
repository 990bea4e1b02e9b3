"""The host code of the layer norm, the 8-bit rows and the checkpoints under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): linear_norm.hip compiled host-only and driven by
tests/sanitize_packed.c, which stands in for the HIP runtime and checks every grid."""
import os

import pytest

from test_linear_norm_sanitizers import CLANG, CLANGXX, HERE, ROOT, SAN_ENV, run


def test_host_side_under_sanitizers(tmp_path):
    if not (os.path.exists(CLANG) and os.path.exists(CLANGXX)):
        pytest.skip("ROCm clang not available")
    obj, lib = tmp_path / "ln_san.o", tmp_path / "libln_san.so"
    csrc = os.path.join(ROOT, "dense_gemm_f16f32_amd", "csrc")
    # host-only compile: no device code is built, the sanitizers apply to the host pass only
    host = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    run([CLANGXX, "-x", "hip", "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g",
         "-std=c++17", "-fPIC", *host, "-Xarch_host", "-fno-sanitize-recover=all",
         "-I", os.path.join(ROOT, "include"), "-I", csrc,
         "-c", os.path.join(csrc, "linear_norm.hip"), "-o", str(obj)])
    run([CLANGXX, "-shared", *host, str(obj), "-o", str(lib)])
    fatbin = [ln.split()[-1] for ln in run(["nm", "-u", str(lib)]).splitlines()
              if "__hip_fatbin" in ln]
    assert len(fatbin) == 1
    exe = tmp_path / "san_packed"
    run([CLANG, "-std=c99", "-O1", "-g", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
         "-fsanitize=undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror",
         "-Wno-unused-function", f"-DFATBIN_SYM={fatbin[0]}",
         "-I", os.path.join(ROOT, "include"), os.path.join(HERE, "sanitize_packed.c"),
         "-L", str(tmp_path), "-lln_san", f"-Wl,-rpath,{tmp_path}", "-rdynamic", "-o", str(exe)])
    out = run([str(exe)], env=SAN_ENV)
    assert out.strip().endswith("ok"), out
