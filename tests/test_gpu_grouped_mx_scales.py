"""GPU: MXFP4 products whose block scales are far apart, at both ends of the
scale byte.  The products are those of scales near 1 times one power of two, so
they and their sums are exact in fp32 and every result is the exact one,
rounded once to bf16."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from oracle.mxfp4 import mxfp4_dequantize
from tests.gpu_common import DEV, host, require_native, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _mx(shape, scale, g):
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.full((*shape[:-1], shape[-1] // 32), scale, device=DEV, dtype=torch.uint8)
    values = torch.from_numpy(mxfp4_dequantize(host(codes), host(scales))).to(DEV)
    return moeq.QWeight(moeq.FMT_MXFP4, *shape, codes, None, scales), values


# E2M1 products are multiples of 1/4 of magnitude 36 at most; the sums of 1056
# of them stay below 2^18 quarters, and x's and w's scales together are 2^(sx + sw - 254).
@pytest.mark.parametrize("sx,sw", [(0, 254), (254, 0), (1, 250), (3, 240), (128, 126), (90, 90), (170, 160), (0, 140)])
@pytest.mark.parametrize("sizes,nout", [([1, 2, 0, 1], 72), ([130, 257, 0, 64] * 10, 2056), ([130, 257, 0, 64], 136)])
def test_scales_at_both_ends(sx, sw, sizes, nout):
    say(f"grouped mxfp4 scales {sx} {sw} {len(sizes)} {nout}")
    g = torch.Generator(device=DEV).manual_seed(8)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    (xq, x), (wq, w) = _mx((1, int(off[-1]), 1056), sx, g), _mx((len(sizes), nout, 1056), sw, g)
    y = moeq.moeq_grouped_mm_mxfp4(xq, wq, torch.from_numpy(off).to(DEV))
    for e in range(len(sizes)):
        lo, hi = int(off[e]), int(off[e + 1])
        want = (x[0, lo:hi] @ w[e].t()).to(torch.bfloat16)
        assert torch.equal(y[lo:hi], want), (e, (y[lo:hi] != want).sum().item())
