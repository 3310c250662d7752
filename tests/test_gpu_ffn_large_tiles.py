"""GPU: the feed-forward block's large tiles and their gradients, at every height
of a tile.  Which kernel runs at
these sizes is checked in test_kernel_choice_cpu.py.

Tolerances are those of test_gpu_ffn.py."""

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from tests.gpu_common import require_native, say
from tests.test_gpu_ffn import _case, _check_backward, _check_forward
from tests.test_gpu_grouped import _untouched
from tests.test_gpu_guarded import Guarded

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
# Rows of an expert: tiles of 1 to 256 rows, one to three of an expert.
SIZES = [100, 180, 250, 256, 700, 64] * 6
SHAPES = [(72, 1000), (520, 264)]   # H, I


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


@pytest.mark.parametrize("H,I", SHAPES)
def test_block_and_gradients(H, I):
    say(f"ffn large tiles H={H} I={I}")
    x, dy, w1, w2, off, doff = _case(SIZES, 3, 2, H, I, seed=3)
    M, E = x.shape[0], len(SIZES)
    y, gu = Guarded((M, H), BF16, 7.0), Guarded((M, 2 * I), F32, 7.0)
    ws = Guarded((moeq.moeq_grouped_ffn_workspace_bytes(M, E, H, I),), U8)
    moeq.moeq_grouped_ffn(x, w1, w2, doff, out=y.t, gu=gu.t, workspace=ws.t)
    for t in (y, gu, ws):
        t.check("forward")
    _check_forward(x, w1, w2, off, y.t, gu.t)
    assert _untouched(y.t, off) and _untouched(gu.t, off)
    plain = moeq.moeq_grouped_ffn(x, w1, w2, doff)      # without saving: the same bits
    assert torch.equal(plain[off[0]:off[-1]], y.t[off[0]:off[-1]])

    gu.t[:off[0]], gu.t[off[-1]:] = float("nan"), float("inf")
    dx, bw = Guarded((M, H), BF16, 7.0), Guarded((moeq.moeq_grouped_ffn_backward_workspace_bytes(M, E, H, I),), U8)
    for dtype, half in ((F32, 2.0 ** -24), (BF16, 2.0 ** -8)):
        dw1, dw2 = Guarded((E, 2 * I, H), dtype), Guarded((E, H, I), dtype)
        grads = moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, doff, gu.t, grad_x=dx.t, grad_gate_up=dw1.t,
                                               grad_down=dw2.t, workspace=bw.t)
        for t in (dx, dw1, dw2, bw):
            t.check("backward")
        _check_backward(dy, x, w1, w2, off, gu.t, grads, half)
        assert _untouched(dx.t, off)
