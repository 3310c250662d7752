"""Build libmoeq.so (the HIP kernels and the C ABI) in-tree for gfx950.

Run ``python -m bit_weight_quantization_moeq_amd.build`` (or call
:func:`build`); the shared library lands next to this file.  Cross-compiles
without a GPU.
"""

import concurrent.futures
import os
import shutil
import subprocess
import sys
import tempfile

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmoeq.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
SOURCES = ["api.hip", "quant.hip", "route.hip", "experts.hip", "decode.hip", "router.hip",
           "api_grouped.hip", "mxfp4.hip", "grouped.hip", "clip.hip",
           "api_ffn.hip", "ffn.hip", "api_fp8.hip", "fp8.hip", "fp8_mm.hip",
           "api_ortho.hip", "ortho.hip"]
ARCH = "gfx950"

# IEEE fp32 division and denormals stay on (no fast-math, no FTZ): the NF4 and
# int8 codes are defined through correctly rounded fp32 arithmetic.  Packed
# fp32 instructions are disabled for all device code.
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc():
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found; ROCm is required to build libmoeq")
    return exe


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"hipcc failed ({proc.returncode}):\n{proc.stdout}\n{proc.stderr}")


def build(verbose=False):
    """Compile every source to an object in parallel, then link."""
    hip = hipcc()
    compile_flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="moeq_build_") as tmpdir:
        objs = [os.path.join(tmpdir, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        cmds = [[hip, *compile_flags, f"-I{INCLUDE}", f"-I{CSRC}", "-c", "-o", o, os.path.join(CSRC, s)]
                for s, o in zip(SOURCES, objs)]
        with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(cmds), os.cpu_count() or 1)) as pool:
            for f in [pool.submit(_run, c, verbose) for c in cmds]:
                f.result()
        tmp = LIB_PATH + ".tmp"
        _run([hip, *FLAGS, "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
