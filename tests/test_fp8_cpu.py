"""Refusals of the FP8 entry points, on the host: the binding's structural
checks on CPU tensors, and the library's own before any HIP call."""

import ctypes
import os

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq

pytestmark = pytest.mark.skipif(not os.path.exists(moeq.library_path()), reason="libmoeq.so not built")
P = ctypes.c_void_p
BF = torch.bfloat16
ROW, TILE = moeq.FMT_FP8_ROW, moeq.FMT_FP8_TILE
FAR = 1 << 40


def _q(fmt, E=2, R=8, C=64):
    return moeq.QWeight.empty(fmt, E, R, C, device="cpu")


def test_layout():
    q = _q(ROW, 2, 130, 272)
    assert q.blocksize == 128 and [s for _, s, _ in q.layout()] == [(2, 130, 272), (2, 130, 3)]
    q.validate_layout()
    t = _q(TILE, 2, 130, 272)
    assert [s for _, s, _ in t.layout()] == [(2, 130, 272), (2, 2, 3)]
    assert t.nbytes() == 2 * 130 * 272 + 2 * 2 * 3 * 4
    assert t.expert(1).validate_layout().shape == (1, 130, 272) and t.like("cpu").validate_layout().format == TILE
    t.scale_codes = torch.empty(1, dtype=torch.uint8)
    with pytest.raises(ValueError):
        t.validate_layout()
    q.qdata = q.qdata.view(torch.uint8)
    with pytest.raises(TypeError):
        q.validate_layout()
    q = _q(ROW, 2, 130, 272)
    q.scales = q.scales[:, :, :2].contiguous()
    with pytest.raises(ValueError):
        q.validate_layout()
    with pytest.raises(ValueError):
        _q(ROW, C=40).validate_layout()


def test_binding_refuses():
    w, off = torch.empty((2, 8, 64), dtype=BF), torch.zeros(3, dtype=torch.int32)
    quant, mm = moeq.moeq_quantize_fp8, moeq.moeq_grouped_mm_fp8
    bad = [
        (ValueError, quant, (torch.empty((2, 8, 40), dtype=BF),), {}),
        (ValueError, quant, (torch.empty(64, dtype=BF),), {}),
        (TypeError, quant, (w.float(),), {}),
        (ValueError, quant, (w.transpose(1, 2),), {}),
        (ValueError, quant, (w, moeq.FMT_MXFP4), {}),
        (ValueError, quant, (w,), dict(out=_q(ROW, R=4))),
        (ValueError, quant, (w,), dict(out=moeq.QWeight.empty(moeq.FMT_MXFP4, 2, 8, 64, device="cpu"))),
        (ValueError, mm, (_q(ROW), _q(TILE), off), {}),                  # x must be one "expert"
        (ValueError, mm, (_q(ROW, 1, 5, 32), _q(TILE), off), {}),        # columns differ
        (ValueError, mm, (_q(TILE, 1), _q(TILE), off), {}),              # tile scales on x
        (ValueError, mm, (_q(ROW, 1), _q(ROW), off), {}),                # row scales on w
        (ValueError, mm, (_q(ROW, 1), _q(TILE), off[:2]), {}),
        (TypeError, mm, (_q(ROW, 1), _q(TILE), off.long()), {}),
        (ValueError, mm, (_q(ROW, 1), _q(TILE), off), dict(out=torch.empty((8, 16), dtype=BF))),
        (TypeError, mm, (w, _q(TILE), off), {}),
        # everything right but on the CPU
        (TypeError, quant, (w,), dict(out=_q(TILE))),
        (TypeError, moeq.moeq_dequantize, (_q(ROW),), {}),
        (TypeError, mm, (_q(ROW, 1), _q(TILE), off), {}),
    ]
    for err, fn, args, kw in bad:
        with pytest.raises(err):
            fn(*args, **kw)


def _qw(fmt=ROW, E=1, R=8, C=64, bs=128, q=FAR, s=2 * FAR, c=0):
    return moeq._QW(fmt, E, R, C, bs, q, s, c)


def test_library_refuses_the_format():
    lib = moeq._load()

    def quant(q, w=3 * FAR):
        return lib.moeq_quantize_fp8(P(w), ctypes.byref(q), None)

    def back(q, out=3 * FAR):
        return lib.moeq_dequantize_fp8(ctypes.byref(q), P(out), None)

    for call in (quant, back):
        for fmt in (0, 1, 2, 3, 4, 7, -1):
            assert call(_qw(fmt=fmt)) == -4
        assert call(_qw(C=40)) == -3 and call(_qw(bs=64)) == -3
        assert call(_qw(E=0)) == -1 and call(_qw(R=0)) == -1 and call(_qw(C=0)) == -1
        assert call(_qw(q=0)) == -1 and call(_qw(s=0)) == -1 and call(_qw(c=FAR)) == -1
        assert call(_qw(q=FAR + 8)) == -5 and call(_qw(s=FAR + 2)) == -5
        assert call(_qw(E=1 << 20, R=1 << 20, C=256)) == -2      # 2^41 blocks
        assert call(_qw(), 0) == -1 and call(_qw(), 3 * FAR + 8) == -5
        # shared memory: the codes, the scales, the last of each
        assert call(_qw(), FAR) == -1 and call(_qw(), 2 * FAR) == -1
        assert call(_qw(), FAR + 8 * 64 - 16) == -1 and call(_qw(s=2 * FAR + 4), 2 * FAR + 32) == -1
    assert quant(_qw(s=FAR + 16)) == -1
    assert lib.moeq_quantize_fp8(P(FAR), None, None) == -1 and lib.moeq_dequantize_fp8(None, P(FAR), None) == -1
    # the calls of the other formats keep refusing it
    assert lib.moeq_quantize_nf4(P(FAR), ctypes.byref(_qw()), None) == -4
    assert lib.moeq_dequantize(ctypes.byref(_qw()), P(FAR), None) == -4
    assert lib.moeq_quantize_mxfp4(P(FAR), ctypes.byref(_qw()), None) == -4
    assert lib.moeq_qweight_copy_async(ctypes.byref(_qw()), ctypes.byref(_qw()), None) == -4


def test_library_refuses_products():
    lib = moeq._load()

    def mm(x=None, w=None, off=5 * FAR, out=6 * FAR):
        x = x or _qw()
        w = w or _qw(TILE, 3, 16, q=3 * FAR, s=4 * FAR)
        return lib.moeq_grouped_mm_fp8(ctypes.byref(x), ctypes.byref(w), P(off), P(out), None)

    assert mm(_qw(TILE)) == -4 and mm(w=_qw(ROW, 3, 16)) == -4 and mm(_qw(fmt=4)) == -4
    assert mm(_qw(E=2)) == -2 and mm(_qw(C=32)) == -2 and mm(w=_qw(TILE, 3, 12)) == -2 and mm(w=_qw(TILE, 1025, 16)) == -2
    assert mm(_qw(C=1 << 11), _qw(TILE, 1, 1 << 19, 1 << 11)) == -2     # N * K * 2 = 2^31
    assert mm(_qw(R=(1 << 28) + 1)) == -2
    assert mm(off=0) == -1 and mm(out=0) == -1 and mm(out=6 * FAR + 8) == -5
    for at in (FAR, 2 * FAR, 3 * FAR, 4 * FAR, 5 * FAR):
        assert mm(out=at) == -1
    assert mm(_qw(R=0, q=0, s=0)) == 0                                    # no rows: a valid no-op
