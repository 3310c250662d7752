"""Grouped products without rows, on the host: a valid no-op of the library
that launches nothing, in MXFP4 as in bf16, and refused where the rest of the
call is wrong."""

import ctypes
import os

import pytest

import bit_weight_quantization_moeq_amd as moeq

pytestmark = pytest.mark.skipif(not os.path.exists(moeq.library_path()), reason="libmoeq.so not built")

P = ctypes.c_void_p


def _qw(E=1, R=0, C=64, q=0, s=0, c=0, bs=32, fmt=moeq.FMT_MXFP4):
    return moeq._QW(fmt, E, R, C, bs, q, s, c)


def _mm(x, w, off=4096, out=4096):
    return moeq._load().moeq_grouped_mm_mxfp4(ctypes.byref(x), ctypes.byref(w), P(off), P(out), None)


def test_mxfp4_product_of_no_rows_is_a_no_op():
    w = _qw(E=3, R=16, q=256, c=1024)
    assert _mm(_qw(), w) == 0
    assert _mm(_qw(), w, off=0, out=0) == 0
    assert _mm(_qw(q=256, c=1024), w) == 0
    # what is wrong apart from that stays refused
    assert _mm(_qw(R=-1), w) == -1
    assert _mm(_qw(E=2), w) == -2
    assert _mm(_qw(C=32), w) == -2
    assert _mm(_qw(bs=64), w) == -3
    assert _mm(_qw(s=512), w) == -1
    assert _mm(_qw(q=8, c=1024), w) == -5
    assert _mm(_qw(R=4), w) == -1                       # rows without data
    assert _mm(_qw(), _qw(E=3, R=0)) == -1              # weights without rows
    assert _mm(_qw(), _qw(E=3, R=12, q=256, c=1024)) == -2


def test_formats_calls_still_refuse_no_rows():
    lib = moeq._load()
    assert lib.moeq_quantize_mxfp4(P(4096), ctypes.byref(_qw(q=256, c=1024)), None) == -1
    assert lib.moeq_dequantize_mxfp4(ctypes.byref(_qw(q=256, c=1024)), P(4096), None) == -1
