"""Builds libgemm_f32.so (the HIP kernels and the C ABI) in-tree for gfx950.

    python -m dense_fp32_gemm_amd.build [--verbose] [--poison-lds]

hipcc compiles for gfx950 only.  Packed-FP32 instruction selection is turned
off for device code (-Xclang -target-feature -Xclang -packed-fp32-ops); the
host pass prints a harmless "not a recognized feature" warning for it.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", f) for f in
           ("gemm_f32.hip", "host.hip", "rows_route.hip", "rows_grouped.hip", "rows_adapters.hip", "ffn_norm.hip",
            "ffn_quantize.hip", "ffn_int8.hip", "ffn_gated.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libgemm_f32.so")
ARCH = "gfx950"

HIPFLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-shared",
    f"--offload-arch={ARCH}",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fvisibility=hidden",
    "-Wall", "-Wno-unused-command-line-argument",
]


# Debug build: -DGEMM_F32_POISON_LDS makes the kernels set every LDS slot to
# NaN before it is refilled or first written (see kPoisonLds in gemm_f32.hip and rows_tile.h),
# so a stale LDS read shows up as NaN in the result (of the row-chosen products, the 8-bit and the gated
# ones: the panels of their K loops; not their lists of row offsets.  8-bit sums cannot hold a NaN: there every
# byte is set, and a stale read gives wrong sums).  gemm_f32_describe() then ends
# with " lds=poisoned".
POISON_LDS = "-DGEMM_F32_POISON_LDS"


def command(out: str, extra: list[str] | None = None, poison_lds: bool = False,
            sources: list[str] | None = None) -> list[str]:
    """The hipcc command line that builds `sources` (all of them: the library) into `out`."""
    flags = [*HIPFLAGS, *([POISON_LDS] if poison_lds else []), *(extra or [])]
    return ["hipcc", *flags, "-I", INCLUDE, *(sources or SOURCES), "-o", out]


def build(verbose: bool = False, extra: list[str] | None = None, poison_lds: bool = False) -> str:
    """Compile the library; returns its path.  Always recompiles.

    The sources compile side by side (they share nothing but host symbols),
    then link.
    """
    tmp = LIBRARY + ".tmp%d" % os.getpid()
    objects = ["%s.%s.o" % (tmp, os.path.basename(src)) for src in SOURCES]
    jobs = []
    noise = "'-packed-fp32-ops' is not a recognized feature for this target"

    def finish(proc):
        out, _ = proc.communicate()
        msgs = [l for l in out.splitlines() if noise not in l and l.strip()]
        if verbose and msgs and proc.returncode == 0:
            print("\n".join(msgs), flush=True)
        return "" if proc.returncode == 0 else "\n".join(msgs)

    def start(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)

    try:
        for src, obj in zip(SOURCES, objects):
            jobs.append(start([*command(obj, extra, poison_lds, [src]), "-c"]))
        errors = [e for e in [finish(j) for j in jobs] if e]
        if not errors:
            errors = [e for e in [finish(start(["hipcc", "-shared", f"--offload-arch={ARCH}", *objects, "-o", tmp]))] if e]
        if errors:
            raise RuntimeError("hipcc failed:\n" + "\n".join(errors))
        os.replace(tmp, LIBRARY)
    finally:
        for obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
    return LIBRARY


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, poison_lds="--poison-lds" in sys.argv)
    print(LIBRARY)
