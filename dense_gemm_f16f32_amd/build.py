"""Compile the HIP library (libgemm_f16f32.so) for gfx950, in-tree.

Every call recompiles.  Flags: -O3 for gfx950 only; packed fp32 arithmetic is disabled
(`-packed-fp32-ops`), so the compiler emits no packed-fp32 vector ops.  After compiling, the
wait states around the inline-asm MFMAs are checked in the built code (check_mfma_waits).
"""
from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "gemm_f16f32.hip")
SO = os.path.join(PKG, "libgemm_f16f32.so")
# The linear layer and the norm (include/linear_norm.h), a library of its own.
LN_SRC = os.path.join(PKG, "csrc", "linear_norm.hip")
LN_SO = os.path.join(PKG, "liblinear_norm.so")
# Its CPython module for torch tensors (host code only).
BINDING_SRC = os.path.join(PKG, "csrc", "torch_binding.cpp")
BINDING_SO = os.path.join(PKG, "_linear_norm.so")
# The matrix-core rate probe (measurement only: bench.py --mfma-ceiling).
PROBE_SRC = os.path.join(PKG, "csrc", "mfma_ceiling.hip")
PROBE_SO = os.path.join(PKG, "libmfma_ceiling.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function"]


LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")

KERNEL_SOURCES = ("gemm_kernels.hpp", "gemm_tiles.hpp")


def strip_comments(text: str) -> str:
    """C++ source without comments and with runs of white space collapsed (the sources have
    no string literals that contain comment markers)."""
    import re
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    text = re.sub(r"//[^\n]*", " ", text)
    return " ".join(text.split())


def kernel_source_hash() -> str:
    """sha256 (first 16 hex digits) of the files that fix the kernels' code -- the device code
    and the tile configurations -- with comments and white space removed, so that only a code
    change counts.  The planner and its dispatch table are left out: they choose the launch
    configuration.  The dispatch table and the HBM-traffic record carry the hash they were
    measured at."""
    import hashlib
    h = hashlib.sha256()
    for name in KERNEL_SOURCES:
        with open(os.path.join(PKG, "csrc", name)) as f:
            h.update(name.encode() + b"\0" + strip_comments(f.read()).encode())
    return h.hexdigest()[:16]

# Kernels whose 16x16x32 MFMAs are inline asm (the 256 x 256 x 64 tile on 2 x 2 wavefronts:
# its DMA, persistent, split-K and generic forms).  The compiler's hazard checks do not see
# those MFMAs, so the code provides the wait states itself (gemm_kernels.hpp, mfma16).
ASM_MFMA_KERNELS = ("mfma_ceiling",                         # the rate probe (both)
                    "lk8lin_ring",                          # the linear layer's 256 x 256 tile
                    "ILi256ELi256ELi64ELi2ELi1ELi2ELi2E",   # gemm_dma*, tile 1
                    "gemm_genericILi256ELi256ELb")          # gemm_generic, 256 x 256 tiles


def _asm_mfma_kernel(name: str) -> bool:
    return any(k in name for k in ASM_MFMA_KERNELS) and (
        "gemm_generic" not in name or "ELi2ELi2ELb" in name)


def disassemble(so_path: str, *options: str) -> str:
    """AMD assembly of the gfx950 code object inside a library built here."""
    import tempfile
    with tempfile.TemporaryDirectory() as d:
        fat, co = os.path.join(d, "fatbin"), os.path.join(d, "gfx950.co")
        # an explicit output file: without one objcopy rewrites its input in place
        subprocess.run(["objcopy", "--dump-section", f".hip_fatbin={fat}", so_path,
                        os.path.join(d, "copy.so")], check=True, capture_output=True)
        subprocess.run([os.path.join(LLVM, "clang-offload-bundler"), "--unbundle", "--type=o",
                        f"--input={fat}", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950",
                        f"--output={co}"], check=True, capture_output=True)
        return subprocess.run([os.path.join(LLVM, "llvm-objdump"), *(options or ("-d",)),
                               "--mcpu=gfx950", co],
                              check=True, capture_output=True, text=True).stdout


def scan_mfma_waits(asm: str):
    """Scans the asm-MFMA kernels of a disassembly, in program order: after an MFMA that
    writes accumulator registers, no v_accvgpr_read/mov may come before the drain (four
    `s_nop 7`, 32 wait states); after a v_accvgpr_write/mov, no MFMA may come before an
    `s_nop 7` (the pin's 8 wait states).  Returns (kernels checked, violations)."""
    import re
    checked, bad = 0, []
    for block in re.split(r"\n(?=[0-9a-f]+ <)", asm):
        m = re.match(r"[0-9a-f]+ <([^>]+)>:", block)
        if not m or not _asm_mfma_kernel(m.group(1)):
            continue
        checked += 1
        mfma_pending = write_pending = False
        nops = 0
        for line in block.splitlines()[1:]:
            ins = line.strip().split("//")[0].strip()
            op = ins.split(" ")[0] if ins else ""
            if op == "s_nop" and ins.endswith(" 7"):
                nops += 1
                write_pending = False
                if nops >= 4:
                    mfma_pending = False
                continue
            nops = 0
            if op.startswith("v_mfma"):
                if write_pending:
                    bad.append(f"{m.group(1)}: MFMA right after an accumulator write: {ins}")
                if ins.split(" ")[1].startswith("a["):
                    mfma_pending = True
            elif op in ("v_accvgpr_read_b32", "v_accvgpr_mov_b32") and mfma_pending:
                bad.append(f"{m.group(1)}: accumulator read before the drain: {ins}")
            if op in ("v_accvgpr_write_b32", "v_accvgpr_mov_b32"):
                write_pending = True
    return checked, bad


def check_mfma_waits(so_path: str) -> int:
    """scan_mfma_waits on a built library; raises on a violation (which would mean the compiler
    moved accumulators around the asm MFMAs) and returns the number of kernels checked."""
    checked, bad = scan_mfma_waits(disassemble(so_path))
    if bad:
        raise RuntimeError("asm MFMA wait states not met:\n" + "\n".join(bad[:20]))
    return checked


def kernels_with_private_arrays(so_path: str) -> list:
    """Kernels of a library built here that keep an array in scratch memory, or in LDS by thread:
    for the latter the compiler has every workgroup read its dispatch packet, which lies in host
    memory (about 0.5 us a workgroup, one after the other)."""
    import re
    text = disassemble(so_path, "-D", "-j", ".rodata")
    found = []
    for block in text.split(".amdhsa_kernel ")[1:]:
        field = dict(re.findall(r"\.amdhsa_(\w+) (\d+)", block.split(".end_amdhsa_kernel")[0]))
        if field["private_segment_fixed_size"] != "0" or field["user_sgpr_dispatch_ptr"] != "0":
            found.append(block.split()[0])
    return found


def _compile(src: str, so: str, extra=(), check=None) -> int:
    """Compiles one library, checks it (with `check`, which raises, as well) and moves it in place;
    returns the number of its kernels whose asm-MFMA wait states were checked.  A library that
    fails leaves the one in place alone."""
    tmp = so + ".tmp"
    cmd = [HIPCC, *FLAGS, *extra, "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(PKG, "csrc"), src, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; that is harmless.
    msgs = [ln for ln in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in ln]
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if msgs:
        print("\n".join(msgs))
    try:
        # Every kernel must have its host launch stub; an undefined one means the host pass
        # dropped a kernel and the library would fail to load.
        nm = subprocess.run(["nm", "-D", "--undefined-only", tmp], capture_output=True, text=True)
        missing = [ln.split()[-1] for ln in nm.stdout.splitlines() if "__device_stub__" in ln]
        if nm.returncode != 0 or missing:
            raise RuntimeError("undefined kernel stubs in the built library: "
                               + ", ".join(missing))
        n = check_mfma_waits(tmp)
        if n == 0:
            raise RuntimeError("no asm-MFMA kernel found to check in the built library")
        if check is not None:
            check(tmp)
    except BaseException:
        os.remove(tmp)
        raise
    os.replace(tmp, so)
    return n


def _refuse_private_arrays(so_path: str) -> None:
    found = kernels_with_private_arrays(so_path)
    if found:
        raise RuntimeError("kernels with arrays in memory: " + ", ".join(found))


def build_linear_norm(extra=()) -> str:
    """Compiles the linear layer and the norm (liblinear_norm.so)."""
    _compile(LN_SRC, LN_SO, extra, _refuse_private_arrays)
    return LN_SO


def build_binding() -> str:
    """Compiles the torch binding against the installed torch and liblinear_norm.so."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    tmp = BINDING_SO + ".tmp"
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(rocm, "include"), BINDING_SRC, "-o", tmp,
           "-L", PKG, "-l:" + os.path.basename(LN_SO), "-L", os.path.join(base, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_hip", "-lc10", "-lc10_hip",
           "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + os.path.join(base, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on the torch binding:\n" + r.stdout + r.stderr)
    os.replace(tmp, BINDING_SO)
    return BINDING_SO


def build(extra=()) -> str:
    """Compiles everything: the fp16 product beside the linear layer and the norm (and their
    binding), then the rate probe."""
    from concurrent.futures import ThreadPoolExecutor

    def layer():
        build_linear_norm(extra)
        build_binding()

    with ThreadPoolExecutor(2) as pool:
        for job in [pool.submit(_compile, SRC, SO, extra), pool.submit(layer)]:
            job.result()
    build_probe()
    return SO


def build_probe() -> str:
    """Compiles the matrix-core rate probe (a library of its own, for bench.py only)."""
    tmp = PROBE_SO + ".tmp"
    r = subprocess.run([HIPCC, *FLAGS, PROBE_SRC, "-o", tmp], capture_output=True, text=True)
    msgs = [ln for ln in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in ln]
    if r.returncode != 0:
        raise RuntimeError("hipcc failed on the probe:\n" + "\n".join(msgs))
    if check_mfma_waits(tmp) != 2:
        os.remove(tmp)
        raise RuntimeError("the probe's two asm-MFMA kernels were not found to check")
    os.replace(tmp, PROBE_SO)
    return PROBE_SO


if __name__ == "__main__":
    print(build())
