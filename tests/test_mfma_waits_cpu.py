"""The grouped-product kernels' gfx950 assembly: no instruction uses the result
of a matrix instruction before its wait states have passed, on any path.

The compiler has been seen to leave those wait states out where the use stands
behind a branch; the results were then those of two matrix instructions
before.  The check walks every path of the control flow from each v_mfma."""

import os
import re
import shutil
import subprocess

import pytest

from bit_weight_quantization_moeq_amd import build

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def _registers(text):
    out = set()
    for kind, lo, hi, kind1, one in re.findall(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        out |= {(kind, i) for i in range(int(lo), int(hi) + 1)} if kind else {(kind1, int(one))}
    return out


def _functions(asm):
    for m in re.finditer(r"\n(_ZN\S+):\s*;[^\n]*\n(.*?)\n\.Lfunc_end", asm, re.S):
        lines, labels = [], {}
        for line in m.group(2).split("\n"):
            line = line.split(";")[0].rstrip()
            label = re.match(r"^(\.L\w+):", line)
            if label:
                labels[label.group(1)] = len(lines)
            elif line.strip() and not line.strip().startswith("."):
                lines.append(line.strip())
        yield m.group(1), lines, labels


def _early_uses(lines, labels):
    def after(i):
        if lines[i].startswith("s_endpgm"):
            return []
        jump = labels.get(lines[i].split()[-1]) if lines[i].startswith(("s_branch", "s_cbranch")) else None
        if lines[i].startswith("s_branch"):
            return [jump]
        return [k for k in (jump, i + 1) if k is not None and k < len(lines)]

    for i, line in enumerate(lines):
        if not line.startswith("v_mfma"):
            continue
        need = 12 if "32x32" in line else 8   # passes (8 or 4) and 4 more
        result = _registers(line.split(None, 1)[1].split(",")[0])
        best, stack = {}, [(k, 0) for k in after(i)]
        while stack:
            k, waited = stack.pop()
            if waited >= need or best.get(k, need) <= waited:
                continue
            best[k] = waited
            use = lines[k]
            if use.startswith("v_mfma"):
                dst, a, b = re.findall(r"[va]\[\d+:\d+\]", use)[:3]
                if (_registers(a) | _registers(b)) & result:
                    yield line, use, waited
                if _registers(dst) & result:
                    continue   # accumulates into it: the hardware waits, and that one is checked itself
            elif use.startswith(("v_", "ds_", "buffer_", "global_", "flat_")):
                if " " in use and _registers(use.split(None, 1)[1]) & result:
                    yield line, use, waited
            cost = int(use.split()[1]) + 1 if use.startswith("s_nop") else 1
            stack += [(n, waited + cost) for n in after(k)]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_matrix_results_are_not_used_early(tmp_path):
    out = str(tmp_path / "grouped.s")
    flags = [f for f in build.FLAGS if f != "-shared"]
    r = subprocess.run([HIPCC, *flags, f"-I{build.INCLUDE}", f"-I{build.CSRC}", "--cuda-device-only", "-S", "-o", out,
                        os.path.join(build.CSRC, "grouped.hip")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = 0
    for name, lines, labels in _functions(open(out).read()):
        seen += sum(x.startswith("v_mfma") for x in lines)
        early = list(_early_uses(lines, labels))
        assert not early, (name, early[:3])
    assert seen > 100


def test_the_check_finds_an_early_use_behind_a_branch():
    lines = ["v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]", "s_cbranch_vccnz .LBB0_2", "s_nop 7",
             "v_accvgpr_read_b32 v8, a0", "s_endpgm", "v_accvgpr_read_b32 v9, a2", "s_endpgm"]
    early = list(_early_uses(lines, {".LBB0_2": 5}))
    assert [(u, w) for _, u, w in early] == [("v_accvgpr_read_b32 v9, a2", 1)]
