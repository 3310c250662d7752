"""GPU: the orthogonalised update in tiles of 128.  Which kernels run at these
sizes is checked in test_kernel_choice_cpu.py.

Tolerances are those of test_gpu_orthogonalize.py."""

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from tests.gpu_common import DEV, require_native, say
from tests.test_gpu_guarded import Guarded
from tests.test_gpu_orthogonalize import _check

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
# Matrices enough for tiles of 128, and too few for tiles of 256.
SHAPES = [(100, 200, 328), (100, 328, 200), (100, 201, 331), (100, 331, 201), (200, 130, 136)]


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_updates(shape, dtype):
    say(f"orthogonalize tiles of 128 {shape} {dtype}")
    g = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).to(dtype)
    out, ws = Guarded(shape, BF16), Guarded((moeq.moeq_orthogonalize_workspace_bytes(*shape),), U8, 0xff)
    moeq.moeq_orthogonalize(g, out=out.t, workspace=ws.t)
    out.check("out")
    ws.check("workspace")
    pick = [0, 17, shape[0] - 1]
    _check(g[pick], out.t[pick])
    for e in pick:   # alone, in tiles of 64: each sum takes the same products in the same order
        assert torch.equal(moeq.moeq_orthogonalize(g[e]), out.t[e])
