"""Which kernels run at the sizes that the tests of single kernels are made for, so
that a later change of a rule cannot leave a kernel without a test.  The
launchers' host code is compiled as it is, with the runtime's entry points taken
down by a driver (no GPU)."""

import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

from tests import test_gpu_ffn_large_tiles as ffn
from tests import test_gpu_fp8_large_tiles as fp8
from tests import test_gpu_orthogonalize_tiles as update

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "bit_weight_quantization_moeq_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CXX = shutil.which("g++")
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC) or not CXX, reason="hipcc or g++ not available")


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """launches("ffn M E H I") -> [(kernel, arguments, workgroups, threads)]."""
    tmp = tmp_path_factory.mktemp("launches")
    sources = [os.path.join(CSRC, f) for f in ("ffn.hip", "fp8_mm.hip", "ortho.hip")] + [os.path.join(HERE, "launches", "driver.hip")]
    objects = [str(tmp / (os.path.basename(s) + ".o")) for s in sources]

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]

    with concurrent.futures.ThreadPoolExecutor(len(sources)) as pool:
        list(pool.map(run, [[HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-fPIC", "-O1", "-std=c++17", "-w",
                             f"-I{ROOT}/include", f"-I{CSRC}", "-c", s, "-o", o] for s, o in zip(sources, objects)]))
    exe = str(tmp / "driver")
    # (the device code itself is not there: nothing is launched)
    run([CXX, *objects, "-Wl,--unresolved-symbols=ignore-all", "-o", exe])

    def ask(line):
        r = subprocess.run([exe], input=line + "\n", capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, (r.returncode, r.stderr)
        out = []
        for part in r.stdout.strip().strip(";").split(";"):
            name, groups, threads = part.rsplit(" ", 2)
            kernel, _, args = name.partition("<")
            args = re.sub(r"\(moeq::\(anonymous namespace\)::\w+\)", "", args.rstrip(">"))
            assert 0 < int(groups) and int(groups) * int(threads) < 2 ** 32
            out.append((kernel, args, int(groups), int(threads)))
        return out

    return ask


@pytest.mark.parametrize("K", fp8.BLOCKS + [400])
def test_large_fp8_tiles(launches, K):
    M, E = sum(fp8.SIZES), len(fp8.SIZES)
    for rows in (M, M + 8):
        assert [k[:2] for k in launches(f"fp8 {rows} {E} {fp8.N} {K}")] == [("fp8_rows_kernel", "4, 2, 4, 8, 2")]


@pytest.mark.parametrize("H,I", ffn.SHAPES)
def test_large_ffn_tiles(launches, H, I):
    M, E = sum(ffn.SIZES) + 5, len(ffn.SIZES)
    assert [k[:2] for k in launches(f"ffn {M} {E} {H} {I}")] == [("glu_kernel", "4, 2, 4, 3, 2")]
    assert [k[:2] for k in launches(f"ffn_backward {M} {E} {H} {I}")] == [("glu_backward_kernel", "4, 2, 2, 4, 3, 2")]


@pytest.mark.parametrize("shape", update.SHAPES)
def test_update_tiles_of_128(launches, shape):
    many = [k[1] for k in launches("orthogonalize {} {} {} 2".format(*shape)) if k[0] == "ortho_kernel"]
    alone = [k[1] for k in launches("orthogonalize 1 {} {} 2".format(*shape[1:])) if k[0] == "ortho_kernel"]
    # two steps of A, the polynomial and the result, the last one's in its own type
    assert [a[0] for a in many] == [a[0] for a in alone] == list("012013")
    assert all(a.endswith(", 2, 2, 2, 2, 2, 2") for a in many), many
    assert all(a.endswith(", 2, 2, 1, 1, 3, 3") for a in alone), alone
