"""The assembly check of test_mfma_waits_cpu.py for the kernels of the
feed-forward block, the FP8 product and the orthogonalised update: no
instruction uses the result of a matrix instruction before its wait states have
passed, on any path.  The 16x16x128 instruction takes as many passes as the
32x32 ones of 16-bit values."""

import os
import re
import subprocess

import pytest

from bit_weight_quantization_moeq_amd import build
from tests.test_mfma_waits_cpu import HIPCC, _functions, _registers

SOURCES = {"ffn.hip": 100, "fp8_mm.hip": 500, "ortho.hip": 100}


def _early(lines, labels):
    """(matrix instruction, use, wait states between them) of every use that comes too soon."""
    def after(i):
        if lines[i].startswith("s_endpgm"):
            return []
        jump = labels.get(lines[i].split()[-1]) if lines[i].startswith(("s_branch", "s_cbranch")) else None
        if lines[i].startswith("s_branch"):
            return [jump]
        return [k for k in (jump, i + 1) if k is not None and k < len(lines)]

    regs = [_registers(line.split(None, 1)[1]) if " " in line else set() for line in lines]
    for i, line in enumerate(lines):
        if not line.startswith("v_mfma"):
            continue
        need = 12 if "32x32" in line or "16x16x128" in line else 8   # passes (8 or 4) and 4 more
        result = _registers(line.split(None, 1)[1].split(",")[0])
        best, stack = {}, [(k, 0) for k in after(i)]
        while stack:
            k, waited = stack.pop()
            if waited >= need or best.get(k, need) <= waited:
                continue
            best[k] = waited
            use = lines[k]
            cost = int(use.split()[1]) + 1 if use.startswith("s_nop") else 1
            if use.startswith("v_mfma"):
                ops = re.findall(r"[va]\[\d+:\d+\]", use)
                if (_registers(ops[1]) | _registers(ops[2])) & result:
                    yield line, use, waited
                if _registers(ops[0]) & result:
                    continue   # its own accumulator: the hardware waits, and that one is checked itself
                # the matrix cores take one of a wave's instructions at a time
                cost = 8 if "32x32" in use or "16x16x128" in use else 4
            elif use.startswith(("v_", "ds_", "buffer_", "global_", "flat_")) and regs[k] & result:
                yield line, use, waited
            stack += [(n, waited + cost) for n in after(k)]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", list(SOURCES))
def test_matrix_results_are_not_used_early(source, tmp_path):
    out = str(tmp_path / "kernels.s")
    flags = [f for f in build.FLAGS if f != "-shared"]
    r = subprocess.run([HIPCC, *flags, f"-I{build.INCLUDE}", f"-I{build.CSRC}", "--cuda-device-only", "-S", "-o", out,
                        os.path.join(build.CSRC, source)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = 0
    for name, lines, labels in _functions(open(out).read()):
        seen += sum(x.startswith("v_mfma") for x in lines)
        early = list(_early(lines, labels))
        assert not early, (name, early[:3])
    assert seen > SOURCES[source]


def test_the_check_counts_the_passes_of_instructions_between():
    a = "v_mfma_scale_f32_16x16x128_f8f6f4 v[0:3], v[8:15], v[16:23], 0, v40, v40 op_sel_hi:[0,0,0]"
    b = a.replace("v[0:3]", "v[4:7]")
    use = "v_fmac_f32_e32 v50, v0, v41"
    assert not list(_early([a, b, "s_nop 3", use, "s_endpgm"], {}))
    assert [w for _, _, w in _early([a, b, "s_nop 2", use, "s_endpgm"], {})] == [11]
    assert [w for _, _, w in _early([a, "s_nop 7", use, "s_endpgm"], {})] == [8]
