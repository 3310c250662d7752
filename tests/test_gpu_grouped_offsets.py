"""GPU: offsets that no routing writes.  They give undefined results, but no
access outside the arrays: every buffer lies between guards that come back
untouched, and inputs hold finite values only inside the arrays."""

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from tests.gpu_common import require_native, say
from tests.test_gpu_guarded import Guarded

pytestmark = pytest.mark.gpu

LOW, HIGH = -(1 << 31), (1 << 31) - 1
M = 600
OFFSETS = {
    "descending": [600, 400, 300, 100, 0],
    "zigzag": [0, 500, 100, 600, 200, 600, 0, 600],
    "all rows, many times": [0, 600] * 40,
    "outside": [-50, 700, -1, 601, HIGH, 10],
    "lowest behind a row": [5, LOW, 600, LOW + 1, 1],
    "extremes": [HIGH, LOW, HIGH, 0, LOW, 300, LOW, HIGH],
    "more than 256 experts": [0, 600, LOW, 7, HIGH] * 60,
}


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


@pytest.mark.parametrize("name", list(OFFSETS))
@pytest.mark.parametrize("N,K", [(16, 96), (64, 32), (264, 288), (512, 1056)])
def test_offsets_that_do_not_ascend_stay_inside(name, N, K):
    say(f"grouped offsets {name} N={N} K={K}")
    E = len(OFFSETS[name]) - 1
    g = torch.Generator(device="cuda").manual_seed(3)
    off = torch.tensor(OFFSETS[name], dtype=torch.int32, device="cuda")
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((E, N, K), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16)
    xq, wq = moeq.moeq_quantize_mxfp4(x), moeq.moeq_quantize_mxfp4(w)
    bf16 = dict(dtype=torch.bfloat16)
    y, ymx, dx = Guarded((M, N), fill=7.0, **bf16), Guarded((M, N), fill=7.0, **bf16), Guarded((M, K), fill=7.0, **bf16)
    dw = Guarded((E, N, K), torch.float32, fill=7.0)
    need = moeq.moeq_grouped_mm_grad_weight_workspace_bytes(M, E, N, K)
    ws = Guarded((max(need, 1),), torch.uint8)
    moeq.moeq_grouped_mm(x, w, off, out=y.t)
    moeq.moeq_grouped_mm_mxfp4(xq, wq, off, out=ymx.t)
    moeq.moeq_grouped_mm_grad_input(dy, w, off, grad_x=dx.t)
    moeq.moeq_grouped_mm_grad_weight(dy, x, off, grad_w=dw.t, workspace=ws.t)
    for b in (y, ymx, dx, dw, ws):
        b.check(name)
    # results come from values inside the arrays, all finite, if undefined
    # (the workspace's partial sums start as the guards' pattern, which is finite too)
    for b in (y, ymx, dx, dw):
        assert bool(torch.isfinite(b.t).all())
