"""GPU: gates and up projections whose product leaves fp32's range while silu(g) u
does not: silu comes first, in the forward pass and in the gradients.

x, grad_out and the first column of down select single values, so that every
result is one value of h, dg or du (or the sum of `repeat` equal ones).
Tolerance: h, dg and du are at most 16 fp32 operations, exp's argument off by
2^-23 |g|, a rounding to bf16, a sum of `repeat` terms, another rounding.  Where
exp(g) is below 2^-126 (g < -87.4) fp32 may hold it as zero, and the results, which
have it as a factor, come out as zeros: off by all of themselves (e^-200 2^66 1e37
200 = 2e-28 is the largest here), and no more."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from oracle.ffn import activation_gradients, hidden
from tests.gpu_common import DEV, require_native, say
from tests.test_gpu_grouped import _f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
PAIRS = [(-1e20, 1e20), (-1e20, -1e20), (-200.0, 1e37), (-1e30, 1e30), (-50.0, 1e30), (3.0, -2.0), (-1e38, 1.0), (100.0, 1e10)]


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _near(got, want, repeat, g, label):
    assert np.isfinite(got).all(), (label, got)
    tol = (2.1 * 2.0 ** -8 + (16 + np.abs(np.where(np.abs(g) < 104, g, 0)) + repeat) * 2.0 ** -23) * np.abs(want) + 1e-30
    tol = tol + np.where(g < -87.4, np.abs(want), 0.0)
    assert np.all(np.abs(got - want) <= tol), (label, got, want)


# (weights past few rows, small tiles, large tiles)
@pytest.mark.parametrize("repeat", [1, 3, 4128])
def test_products_past_the_range(repeat):
    say(f"ffn far products repeat={repeat}")
    x = torch.eye(8, device=DEV).to(BF16).repeat(repeat, 1)
    w1 = torch.zeros((1, 16, 8), device=DEV)
    w1[0, 0], w1[0, 8] = torch.tensor(PAIRS, device=DEV).t()
    w1 = w1.to(BF16)
    w2 = torch.zeros((1, 8, 8), dtype=BF16, device=DEV)
    w2[0, :, 0] = 1.0
    off = torch.tensor([0, 8 * repeat], dtype=torch.int32, device=DEV)
    y, gu = moeq.moeq_grouped_ffn(x, w1, w2, off, save=True)
    p = _f64(gu)
    assert np.array_equal(p[:, [0, 8]], np.tile(_f64(w1)[0, [0, 8]].T, (repeat, 1)))
    h = hidden(p)[:, 0]
    _near(_f64(y), np.repeat(h[:, None], 8, 1), 1, p[:, :1], "out")

    scale = 2.0 ** 66   # (its product with u leaves the range, too)
    dy = x * scale
    want = activation_gradients(np.full((8, 1), scale), p[:8][:, [0, 8]])
    for dtype in (F32, BF16):
        _, dw1, dw2 = moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, off, gu, dtype=dtype)
        _near(_f64(dw1)[0, 0], repeat * want[:, 0], repeat, p[:8, 0], "dg")
        _near(_f64(dw1)[0, 8], repeat * want[:, 1], repeat, p[:8, 0], "du")
        _near(_f64(dw2)[0, :, 0], repeat * scale * h[:8], repeat, p[:8, 0], "grad_down")
