"""The linear layer's and the norm's host code at the largest extents it accepts (CPU only):
linear_norm.hip compiled host-only and driven by tests/limits_linear_norm.c, whose stand-in for
the runtime refuses grids of 2^32 threads, as the runtime does."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CLANG = os.path.join(ROCM, "llvm", "bin", "clang")


def run(*cmd):
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, " ".join(map(str, cmd)) + "\n" + r.stdout + r.stderr
    return r.stdout


def test_largest_extents(tmp_path):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang not available")
    csrc = os.path.join(ROOT, "dense_gemm_f16f32_amd", "csrc")
    lib, exe = str(tmp_path / "libln_host.so"), str(tmp_path / "limits")
    # host-only compile: no device code is built
    run(CLANG + "++", "-x", "hip", "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17",
        "-fPIC", "-shared", "-nogpulib", "-I", os.path.join(ROOT, "include"), "-I", csrc,
        os.path.join(csrc, "linear_norm.hip"), "-o", lib)
    fatbin = [ln.split()[-1] for ln in run("nm", "-u", lib).splitlines() if "__hip_fatbin" in ln]
    assert len(fatbin) == 1, fatbin
    run(CLANG, "-std=c99", "-O1", f"-DFATBIN_SYM={fatbin[0]}", "-I", os.path.join(ROOT, "include"),
        os.path.join(HERE, "limits_linear_norm.c"), "-L", str(tmp_path), "-lln_host",
        f"-Wl,-rpath,{tmp_path}", "-rdynamic", "-o", exe)
    assert run(exe).strip().endswith("ok")
