"""The FP8 oracle: E4M3 by hand and against torch's type, exact rational
quotients for the codes."""

from fractions import Fraction

import numpy as np
import torch

from oracle.fp8 import e4m3_decode, e4m3_encode, e4m3_levels, fp8_quantize, fp8_values
from tests.exact import frac, rn32


def _bits(x):
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_levels():
    lv = e4m3_levels()
    assert lv[0] == 0 and lv[1] == 2.0 ** -9 and lv[7] == 7 * 2.0 ** -9 and lv[8] == 2.0 ** -6 and lv[126] == 448
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes.view(np.int8)).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3_decode(codes), ref, equal_nan=True)


def test_encode_rounds_half_to_even():
    lv = e4m3_levels()
    assert np.array_equal(e4m3_encode(lv), np.arange(127))
    mid = (lv[1:] + lv[:-1]) / 2
    want = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(e4m3_encode(mid), want)
    assert np.array_equal(e4m3_encode(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(e4m3_encode(-np.nextafter(mid, 1e9)), np.arange(1, 127) | 128)
    assert e4m3_encode(np.array([-0.0]))[0] == 128


def test_quantize_is_the_nearest_code_of_the_exact_quotient():
    r = np.random.default_rng(0)
    for rows, shape in ((1, (2, 3, 144)), (128, (1, 130, 160))):
        bits = _bits(r.standard_normal(shape) * 10.0 ** r.uniform(-6, 6, shape[:2] + (1,)))
        codes, scales = fp8_quantize(bits, rows)
        w = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).double().numpy()
        lv = [frac(v) for v in e4m3_levels()]
        for e, i, j in [(e, i, j) for e in range(shape[0]) for i in range(0, shape[1], 17) for j in range(0, shape[2], 5)]:
            i0, j0 = i // rows * rows, j // 128 * 128
            top = np.abs(w[e, i0:i0 + rows, j0:j0 + 128]).max()
            assert scales[e, i // rows, j // 128] == rn32(frac(top) / 448)
            q = abs(frac(w[e, i, j])) * 448 / frac(top)
            d = [abs(q - v) for v in lv]
            best = [c for c in range(127) if d[c] == min(d)]
            c = codes[e, i, j]
            assert (c & 127) == (best[0] if len(best) == 1 else [b for b in best if b % 2 == 0][0])
            assert bool(c & 128) == (w[e, i, j] < 0)


def test_zero_and_bad_blocks():
    w = np.zeros((1, 2, 256), np.float32)
    w[0, 0, 3], w[0, 1, 200] = np.inf, -1.0
    codes, scales = fp8_quantize(_bits(w), 1)
    assert np.isnan(scales[0, 0, 0]) and scales[0, 0, 1] == 0 and scales[0, 1, 1] == np.float32(1) / np.float32(448)
    assert not codes[0, 0].any() and codes[0, 1, 200] == 126 | 128
    v = fp8_values(codes, scales, 1)
    assert np.isnan(v[0, 0, :128]).all() and not v[0, 0, 128:].any()
    assert Fraction(float(v[0, 1, 200])) == -448 * Fraction(float(scales[0, 1, 1]))
