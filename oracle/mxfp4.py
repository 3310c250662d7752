"""MXFP4 in 64 bits: 32 consecutive columns share a power-of-two scale, each
value is E2M1 (OCP Microscaling specification, MXFP4)."""

import numpy as np

from .bf16 import bf16_to_f32

BLOCK = 32
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mxfp4_quantize(bits):
    """uint16 bf16 patterns [..., C] -> (codes uint8 [..., C/2], scales uint8
    [..., C/32]).  The even column takes the low nibble."""
    w = bf16_to_f32(np.asarray(bits, np.uint16)).astype(np.float64)
    b = w.reshape(*w.shape[:-1], w.shape[-1] // BLOCK, BLOCK)
    finite = np.isfinite(b).all(-1)
    top = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1), 0.0)
    exp = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1, -1000)   # floor(log2(top))
    s = np.maximum(exp - 2, -127)
    with np.errstate(invalid="ignore"):
        v = np.abs(b) * np.exp2(-s.astype(np.float64))[..., None]
    # nearest level; of two at the same distance the one with the even index
    d = np.abs(np.where(finite[..., None], v, 0.0)[..., None] - LEVELS)
    near = d == d.min(-1, keepdims=True)
    code = np.where(near & (np.arange(8) % 2 == 0), 2, near).argmax(-1).astype(np.uint8)
    code |= np.signbit(b).astype(np.uint8) << 3
    code = np.where(finite[..., None], code, 0).reshape(*w.shape[:-1], w.shape[-1] // 2, 2).astype(np.uint8)
    return code[..., 0] | (code[..., 1] << 4), np.where(finite, s + 127, 255).astype(np.uint8)


def mxfp4_dequantize(codes, scales):
    """Values in fp64: E2M1 value * 2^(scale - 127), NaN for scale 255."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(c >= 8, -1.0, 1.0) * LEVELS[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, BLOCK, -1)
