"""The MXFP4 oracle against exact rational arithmetic, hand-worked blocks and
properties of the format."""

from fractions import Fraction

import numpy as np
import pytest

from oracle.bf16 import bf16_to_f32, f32_to_bf16
from oracle.mxfp4 import LEVELS, mxfp4_dequantize, mxfp4_quantize


def _unpack(codes):
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)


def _bits(v):
    return f32_to_bf16(np.asarray(v, np.float32))


def test_levels_are_e2m1():
    for i, v in enumerate(LEVELS):
        e, f = i >> 1, i & 1
        assert Fraction(float(v)) == (Fraction(f, 2) if e == 0 else Fraction(2) ** (e - 1) * (1 + Fraction(f, 2)))


def test_hand_worked_block():
    v = np.zeros(32)
    v[:10] = [6.0, -3.0, 5.0, 2.5, 3.5, 0.25, 0.75, -1.25, 1.75, 7.5]   # max 7.5: scale 2^0; ties to the even code
    codes, s = mxfp4_quantize(_bits(v))
    assert s.tolist() == [127]
    assert _unpack(codes)[:10].tolist() == [7, 13, 6, 4, 6, 0, 2, 10, 4, 7]
    assert codes[0] == 7 | 13 << 4   # even column in the low nibble


@pytest.mark.parametrize("shift", [-126, -100, -3, 0, 5, 120])
def test_scaling_a_block_by_a_power_of_two_moves_the_scale_alone(shift):
    rng = np.random.default_rng(3)
    base = rng.integers(-255, 256, (16, 32)).astype(np.float64)   # 8-bit integers: exact in bf16
    base[:, 0] = 129
    c0, s0 = mxfp4_quantize(_bits(base))
    c1, s1 = mxfp4_quantize(_bits(base * 2.0 ** shift))
    assert np.array_equal(c0, c1) and np.array_equal(s0.astype(int) + shift, s1.astype(int))


def test_nearest_value_in_exact_arithmetic():
    rng = np.random.default_rng(4)
    bits = _bits(rng.standard_normal((50, 32)) * np.exp2(rng.integers(-40, 40, (50, 1))))
    codes, s = mxfp4_quantize(bits)
    w, c = bf16_to_f32(bits).astype(np.float64), _unpack(codes)
    for i in range(50):
        scale = Fraction(2) ** (int(s[i, 0]) - 127)
        top = max(abs(Fraction(float(v))) for v in w[i])
        assert 4 * scale <= top < 8 * scale
        for j in range(32):
            v = abs(Fraction(float(w[i, j]))) / scale
            got = abs(v - Fraction(float(LEVELS[c[i, j] & 7])))
            assert got == min(abs(v - Fraction(float(x))) for x in LEVELS)
            assert (c[i, j] >> 3) == (w[i, j] < 0)


def test_round_trip_is_idempotent_and_special_blocks():
    rng = np.random.default_rng(5)
    codes, s = mxfp4_quantize(_bits(rng.standard_normal((20, 64))))
    again = mxfp4_quantize(_bits(mxfp4_dequantize(codes, s)))
    assert np.array_equal(mxfp4_dequantize(*again), mxfp4_dequantize(codes, s))
    v = np.zeros((3, 32), np.float32)
    v[1, 3], v[2, 5] = np.inf, np.nan
    codes, s = mxfp4_quantize(_bits(v))
    assert s[:, 0].tolist() == [0, 255, 255] and not codes.any()
    d = mxfp4_dequantize(codes, s)
    assert not d[0].any() and np.isnan(d[1:]).all()


def test_smallest_scale_and_subnormals():
    bits = np.zeros((1, 32), np.uint16)
    bits[0, :4] = [1, 64, 0x8020, 0x007f]   # subnormal bf16: multiples of 2^-133
    codes, s = mxfp4_quantize(bits)
    # scale 2^-127: 1/64 -> 0, 1 -> 1, -0.5 -> -0.5, 127/64 -> 2
    assert s[0, 0] == 0 and _unpack(codes)[0, :4].tolist() == [0, 2, 9, 4]
