"""The linear layer's and the norm's host code under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): linear_norm.hip compiled host-only and driven by
tests/sanitize_linear_norm.c, which stands in for the HIP runtime and checks every grid."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CLANG = os.path.join(ROCM, "llvm", "bin", "clang")
CLANGXX = os.path.join(ROCM, "llvm", "bin", "clang++")
SAN_ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1")


def run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600, **kw)
    assert r.returncode == 0, " ".join(map(str, cmd)) + "\n" + r.stdout + r.stderr
    return r.stdout


def test_linear_norm_host_side_under_sanitizers(tmp_path):
    if not (os.path.exists(CLANG) and os.path.exists(CLANGXX)):
        pytest.skip("ROCm clang not available")
    obj, lib = tmp_path / "ln_san.o", tmp_path / "libln_san.so"
    csrc = os.path.join(ROOT, "dense_gemm_f16f32_amd", "csrc")
    # host-only compile: no device code is built, the sanitizers apply to the host pass only
    run([CLANGXX, "-x", "hip", "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g",
         "-std=c++17", "-fPIC",
         "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
         "-Xarch_host", "-fno-sanitize-recover=all",
         "-I", os.path.join(ROOT, "include"), "-I", csrc,
         "-c", os.path.join(csrc, "linear_norm.hip"), "-o", str(obj)])
    run([CLANGXX, "-shared", "-Xarch_host", "-fsanitize=address",
         "-Xarch_host", "-fsanitize=undefined", str(obj), "-o", str(lib)])
    undefined = run(["nm", "-u", str(lib)])
    fatbin = [ln.split()[-1] for ln in undefined.splitlines() if "__hip_fatbin" in ln]
    assert len(fatbin) == 1, undefined
    exe = tmp_path / "san_ln"
    run([CLANG, "-std=c99", "-O1", "-g", "-fsanitize=address,undefined",
         "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror", f"-DFATBIN_SYM={fatbin[0]}",
         "-I", os.path.join(ROOT, "include"), os.path.join(HERE, "sanitize_linear_norm.c"),
         "-L", str(tmp_path), "-lln_san", f"-Wl,-rpath,{tmp_path}", "-rdynamic", "-o", str(exe)])
    out = run([str(exe)], env=SAN_ENV)
    assert out.strip().endswith("ok"), out
