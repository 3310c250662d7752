"""GPU: the FP8 product's large tiles, at every height of a tile and with one to
ten blocks of the contraction.  Which kernel runs at
these sizes is checked in test_kernel_choice_cpu.py.

Tolerances are those of test_gpu_fp8.py."""

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from oracle.grouped import grouped_mm
from tests.gpu_common import DEV, require_native, say
from tests.test_gpu_fp8 import F8, _check_product, _operands, _values
from tests.test_gpu_grouped import _offsets, _untouched
from tests.test_gpu_guarded import Guarded

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
# Rows of an expert: tiles of 1 to 256 rows, one to three of an expert.
SIZES = [100, 180, 250, 256, 700, 64] * 6
N, BLOCKS = 1000, [112, 128, 256, 384, 512, 640, 1168]   # contractions of 1 to 5 and of 10 blocks


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


@pytest.mark.parametrize("K", BLOCKS)
def test_exact_operands(K):
    """Integer values with scales of powers of two: every sum is an integer below
    2^24 times a power of two, so the result is the exact one, rounded."""
    say(f"fp8 large tiles exact K={K}")
    g = torch.Generator(device=DEV).manual_seed(K)
    off, E = _offsets(SIZES), len(SIZES)
    M, kb, nb = int(off[-1]), -(-K // 128), -(-N // 128)
    xc = torch.randint(-4, 5, (1, M, K), generator=g, device=DEV).float()
    wc = torch.randint(-4, 5, (E, N, K), generator=g, device=DEV).float()
    xs = torch.exp2(torch.randint(-2, 3, (1, M, kb), generator=g, device=DEV).float())
    ws = torch.exp2(torch.randint(-2, 3, (E, nb, kb), generator=g, device=DEV).float())
    xq = moeq.QWeight(moeq.FMT_FP8_ROW, 1, M, K, xc.to(F8), xs)
    wq = moeq.QWeight(moeq.FMT_FP8_TILE, E, N, K, wc.to(F8), ws)
    y = Guarded((M, N), BF16)
    moeq.moeq_grouped_mm_fp8(xq, wq, torch.from_numpy(off).to(DEV), out=y.t)
    y.check("out")
    a, b = _values(xq, wq, [0, M])
    want = torch.from_numpy(grouped_mm(a, b, off.tolist())).to(BF16)   # (exact in fp32 and below, then one rounding)
    assert torch.equal(y.t.cpu(), want)


@pytest.mark.parametrize("K", [400, 1168])
def test_product(K):
    say(f"fp8 large tiles K={K}")
    xq, wq, off, doff = _operands(SIZES, 3, 5, N, K, seed=1)
    y = torch.full((xq.rows, N), 7.0, dtype=BF16, device=DEV)
    moeq.moeq_grouped_mm_fp8(xq, wq, doff, out=y)
    _check_product(y, xq, wq, off)
    assert _untouched(y, off)


def test_nan_blocks():
    """A NaN scale reaches the outputs of its row, or of its columns and expert, alone."""
    say("fp8 large tiles NaN")
    xq, wq, off, doff = _operands(SIZES, 0, 0, N, 400, seed=2)
    row = int(off[4]) + 300
    xq.scales[0, row, 2] = float("nan")
    wq.scales[3, 1, 1] = float("nan")
    y = moeq.moeq_grouped_mm_fp8(xq, wq, doff)
    want = torch.zeros((xq.rows, N), dtype=torch.bool)
    want[row], want[off[3]:off[4], 128:256] = True, True
    assert torch.equal(y.isnan().cpu(), want)
