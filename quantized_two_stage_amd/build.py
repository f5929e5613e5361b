"""Build libqr.so (the HIP kernels and the C ABI of include/qr.h,
include/qr_layer.h and include/qr_f8.h) for gfx950, and libqr_pattern.so, the benchmark's
access-pattern reference (not part of the library's ABI).

Flags that matter for the numerics: -ffp-contract=off (no fused multiply-add
the source does not ask for), no fast-math (IEEE division and denormals);
packed fp32 instructions are disabled for the device code.
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libqr.so")
SOURCES = [os.path.join(CSRC, f) for f in
           ("qr_kernels.hip", "qr_rows.hip", "qr_gemm.hip", "qr_rows_f8.hip", "qr_gemm_f8.hip",
            "qr_experts.hip", "qr_api.cpp", "qr_layer_api.cpp", "qr_f8_api.cpp")]
PATTERN_LIB = os.path.join(PKG, "libqr_pattern.so")
PATTERN_SOURCES = [os.path.join(CSRC, "qr_pattern.hip")]
ARCH = os.environ.get("QR_OFFLOAD_ARCH", "gfx950")

FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-shared",
         "-ffp-contract=off", "-fno-fast-math",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def build(out=LIB, extra=(), verbose=False, sources=SOURCES):
    """Compile the library into `out` (its sources side by side); returns its
    path."""
    tmp = out + ".tmp%d" % os.getpid()

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("hipcc failed (%d)" % res.returncode)

    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(f) + ".o") for f in sources]
        compile_flags = [f for f in FLAGS if f != "-shared"]
        with ThreadPoolExecutor(min(len(sources), os.cpu_count() or 1)) as pool:
            list(pool.map(lambda fo: run(["hipcc", *compile_flags, *extra, "-c", fo[0], "-o",
                                          fo[1]]), zip(sources, objs)))
        run(["hipcc", *FLAGS, *extra, *objs, "-o", tmp])
    os.replace(tmp, out)
    return out


def build_pattern(verbose=False):
    """the benchmark's access-pattern reference library"""
    return build(out=PATTERN_LIB, verbose=verbose, sources=PATTERN_SOURCES)


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_pattern(verbose=True))
