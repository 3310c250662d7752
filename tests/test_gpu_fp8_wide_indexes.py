"""GPU: FP8 tensors of more than 2^31 blocks and 2^31 groups of 16 values, whose
kernels count in 64 bits: every code, scale and value as in a small tensor that
they repeat."""

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from tests.gpu_common import DEV, require_native, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [moeq.FMT_FP8_ROW, moeq.FMT_FP8_TILE])
def test_more_than_2_to_the_31_blocks(fmt):
    require_native()
    say(f"fp8 past 2^31 blocks, format {fmt}")
    # two experts of 2^30 + 2^14 rows of 16 columns, 2^14 rows over and over
    period, turns, C = 1 << 14, (1 << 16) + 1, 16
    one = torch.randn((period, C), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    one[:, 0] *= torch.exp2((torch.arange(period, device=DEV) % 23).float())
    small = moeq.moeq_quantize_fp8(one, fmt)
    w = one.expand(2, turns, period, C).reshape(2, turns * period, C)
    q = moeq.moeq_quantize_fp8(w, fmt)
    del w
    codes = q.qdata.view(torch.uint8).view(2 * turns, -1)
    scales = q.scales.view(2 * turns, -1)
    want = small.qdata.view(torch.uint8).view(1, -1)
    step = 4096
    for i in range(0, 2 * turns, step):
        assert bool((codes[i:i + step] == want).all()), i
        assert bool((scales[i:i + step] == small.scales.view(1, -1)).all()), i
    back = moeq.moeq_dequantize(q).view(2 * turns, -1)
    want = moeq.moeq_dequantize(small).view(1, -1)
    for i in range(0, 2 * turns, step):
        assert bool((back[i:i + step] == want).all()), i
    del back, codes, scales, q
    torch.cuda.empty_cache()
