"""GPU: coefficients of any size, as long as the singular values stay in range:
the polynomial a I + b A + c A A, whose entries a direction without a singular
value raises to a, has to fit the working matrices whatever a, b and c are."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from tests.gpu_common import DEV, require_native, say
from tests.test_gpu_grouped import _f64
from tests.test_gpu_orthogonalize import _check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


@pytest.mark.parametrize("a", [1.0, 200.0, 256.0, 300.0])
@pytest.mark.parametrize("shape", [(1504, 1600), (1600, 1499)])
def test_a_multiple(shape, a):
    """(a, 0, 0) is a G / |G|.  a's products with powers of two are exact, so X's
    rounding to fp16 (2^-11, and 2^-25 of the 2^5 that X is stored with) and the
    output's are all there is, and a few units of fp32.  The largest singular value
    is about 2 a / sqrt(1500)."""
    say(f"orthogonalize multiple {shape} a={a}")
    g = torch.randn((1, *shape), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    x = _f64(g)
    want = a * x / np.sqrt((x * x).sum())
    got = _f64(moeq.moeq_orthogonalize(g, 1, (a, 0.0, 0.0)))
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * np.abs(want) + a * 2.0 ** -30)


# (matrices of few rows, in registers; tiles)
@pytest.mark.parametrize("shape", [(2, 16, 72), (2, 72, 16), (2, 30, 300), (2, 40, 72), (2, 72, 40), (1, 130, 264)])
@pytest.mark.parametrize("table", [[(300.0, -600.0, 301.0)], [(3.0, -4.0, 2.0), (300.0, -600.0, 301.0), (1.5, -0.5, 0.0)],
                                   [(500.0, 10.0, -509.0)], [(100.0, -50.0, -48.0)]])
def test_one_direction(shape, table):
    """One direction along an axis: its singular value goes from 1 to near 1, and
    the directions that the matrix lacks meet a alone."""
    say(f"orthogonalize one direction {shape} {table}")
    for dtype in (F32, BF16):
        g = torch.zeros(shape, dtype=dtype, device=DEV)
        g[:, 3, 5] = 2.0
        _check(g, moeq.moeq_orthogonalize(g, len(table), table), table)


@pytest.mark.parametrize("shape", [(2, 16, 72), (2, 72, 16), (2, 40, 72), (2, 72, 40)])
@pytest.mark.parametrize("table", [[(15.5, 0.0, 0.0), (0.0625, 0.0, 0.0)], [(15.5, 0.0, 0.0), (1.0, -0.004, 0.0)],
                                   [(1.0, 7.0, 7.5), (0.5, -0.002, 0.0)]])
def test_near_the_largest_singular_value(shape, table):
    """One singular value at 15.5, next to the documented 15.9: A holds 15.5^2 2^8."""
    say(f"orthogonalize 15.5 {shape} {table}")
    g = torch.zeros(shape, device=DEV)
    g[:, 3, 5] = 2.0
    _check(g, moeq.moeq_orthogonalize(g, 2, table), table)


@pytest.mark.parametrize("shape", [(2, 20, 200), (2, 72, 200)])
def test_small_and_large_in_turn(shape):
    """Each step has a power of two of its own."""
    say(f"orthogonalize coefficients in turn {shape}")
    g = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(BF16)
    for large in ((240.0, 0.0, 0.0), (240.0, -300.0, 100.0)):
        table = [(0.0625, 0.0, 0.0), large, (0.5, 0.0, 0.0)]
        _check(g, moeq.moeq_orthogonalize(g, 3, table), table)


@pytest.mark.parametrize("shape", [(2, 20, 200), (2, 200, 20), (2, 40, 72)])
def test_as_many_steps_as_there_may_be(shape):
    """64 steps, the last with coefficients of its own."""
    say(f"orthogonalize 64 steps {shape}")
    g = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)
    table = [(1.5, -0.5, 0.0)] * 63 + [(200.0, -300.0, 110.0)]
    _check(g, moeq.moeq_orthogonalize(g, 64, table), table)
