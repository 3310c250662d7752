"""FP8 (E4M3: sign, four exponent bits, three fraction bits, largest 448) with
a scale for each block of 128, in 64 bits."""

import numpy as np

from .bf16 import bf16_to_f32

BLOCK = 128
MAX = 448.0


def e4m3_levels():
    """The 127 magnitudes of codes 0 .. 126, ascending."""
    c = np.arange(127)
    e, f = c >> 3, c & 7
    return np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * np.exp2(e - 7.0))


def e4m3_decode(codes):
    c = np.asarray(codes, np.uint8)
    v = np.append(e4m3_levels(), np.nan)[c & 127]
    return np.where(c & 128, -v, v)


def e4m3_encode(v):
    """Nearest code to |v| <= 448, ties to the even code."""
    lv = e4m3_levels()
    a = np.abs(v)
    hi = np.clip(np.searchsorted(lv, a), 1, 126)
    lo = hi - 1
    up, down = lv[hi] - a, a - lv[lo]   # (exact: neighbours differ by a power of two)
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _spread(s, rows, R, C):
    """Block values [..., nr, nc] at each of [..., R, C]."""
    return np.repeat(np.repeat(s, rows, -2)[..., :R, :], BLOCK, -1)[..., :C]


def fp8_quantize(bits, rows):
    """uint16 bf16 patterns [E, R, C] -> (codes uint8 [E, R, C], scales fp32 [E,
    ceil(R / rows), ceil(C / 128)]), a scale for each `rows` rows by 128 columns."""
    w = bf16_to_f32(np.asarray(bits, np.uint16)).astype(np.float64)
    E, R, C = w.shape
    nr, nc = -(-R // rows), -(-C // BLOCK)
    full = np.zeros((E, nr * rows, nc * BLOCK))
    full[:, :R, :C] = np.abs(w)
    top = full.reshape(E, nr, rows, nc, BLOCK).max((2, 4))
    ok = np.isfinite(full).reshape(E, nr, rows, nc, BLOCK).all((2, 4))
    top = np.where(ok, top, 0.0)
    scale = np.where(ok, np.float32(top) / np.float32(MAX), np.float32("nan")).astype(np.float32)
    each, fine = _spread(top, rows, R, C), _spread(ok, rows, R, C)
    v = np.where(fine, w, 0.0) * MAX / np.where(each > 0, each, 1.0)
    return np.where(fine, e4m3_encode(v), 0).astype(np.uint8), scale


def fp8_values(codes, scales, rows):
    """code * scale in 64 bits, [E, R, C]."""
    return e4m3_decode(codes) * _spread(np.asarray(scales, np.float64), rows, *np.shape(codes)[-2:])
