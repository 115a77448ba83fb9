"""Builds libpgemm.so (gfx950) in-tree with hipcc.

    python -m software_pipelined_tiled_pgemm_amd.build [--verbose] [--poison-lds]

Flags: -O3; packed-fp32 instructions disabled; fp32 denormals kept (the
streaming kernels must match IEEE binary32 bit for bit); no fast-math;
explicit kernel arguments preloaded into SGPRs.
Each source is compiled to an object (PER_FILE adds flags to single
sources), then the objects are linked into the shared library.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libpgemm.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

OBJDIR = os.path.join(PKG, "_build")

FLAGS = [
    "--offload-arch=" + ARCH,
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fno-gpu-flush-denormals-to-zero",
    "-fno-fast-math",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-Wall",
    # The explicit kernel arguments arrive preloaded in SGPRs instead of
    # through a scalar load at the start of every wave (measured: 256^3 GEMM
    # 4.94 -> 4.59 us per launch, large shapes unchanged).
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
]

# Extra code-generation flags of single sources.
PER_FILE = {
    # The 16x16x32 GEMM kernels: MFMA results in ordinary VGPRs (without it
    # the compiler moves accumulator blocks between register files inside
    # the K loop; see the file's header comment).
    "gemm_f16_m16.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    # The layer operators' products are the same kernels with other
    # operand layouts and epilogues.
    "linear.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "layer_split.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "ffn.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "xent.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
}


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(ln for ln in (res.stdout + res.stderr).splitlines()
                    if "packed-fp32-ops" not in ln)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed (%d):\n%s" % (res.returncode, out))
    if verbose and out.strip():
        print(out)


def build(verbose: bool = False, extra_flags=None) -> str:
    """Compile every HIP source and link libpgemm.so (always recompiles)."""
    from concurrent.futures import ThreadPoolExecutor

    os.makedirs(OBJDIR, exist_ok=True)
    tag = ".%d" % os.getpid()
    jobs = []
    for src in sources():
        name = os.path.basename(src)
        obj = os.path.join(OBJDIR, name + tag + ".o")
        cmd = ([HIPCC] + FLAGS + PER_FILE.get(name, []) + list(extra_flags or [])
               + ["-c", src, "-o", obj])
        jobs.append((cmd, obj))
    objs = [o for _, o in jobs]
    tmp = LIB + ".tmp%d" % os.getpid()
    try:
        with ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            list(ex.map(lambda j: _run(j[0], verbose), jobs))
        _run([HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC"] + objs + ["-o", tmp], verbose)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    # --poison-lds: the race-detection build (released LDS stages filled with
    # NaN behind an extra barrier); for test runs only, never the product.
    build(verbose="--verbose" in sys.argv,
          extra_flags=["-DPGEMM_POISON_LDS=1"] if "--poison-lds" in sys.argv else None)
    print(LIB)
