"""The host code of the feed-forward block, the FP8 format and the
orthogonalised update built with AddressSanitizer and
UndefinedBehaviorSanitizer (host code only; no GPU): a driver with its own
expectations, which exits non-zero on an unexpected result or a sanitizer
report."""

import os
import shutil
import subprocess

import pytest

from tests.test_grouped_sanitized_cpu import CSRC, HERE, ROOT


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="hipcc not available")
def test_training_host_code_under_sanitizers(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    exe = str(tmp_path / "driver")
    sources = [os.path.join(CSRC, f) for f in ("api_grouped.hip", "api_ffn.hip", "api_fp8.hip", "api_ortho.hip")]
    cmd = [hipcc, "--offload-arch=gfx950", "-x", "hip",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-g", "-O1", "-std=c++17", f"-I{ROOT}/include", f"-I{CSRC}",
           "-w", *sources, os.path.join(HERE, "training_driver.hip"), "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "all checks passed" in r.stdout
