"""Results that share memory with an operand, on the host: refused before any
device call, since workgroups read operands while others store results."""

import array
import ctypes
import os

import pytest

import bit_weight_quantization_moeq_amd as moeq

pytestmark = pytest.mark.skipif(not os.path.exists(moeq.library_path()), reason="libmoeq.so not built")

P = ctypes.c_void_p
MB = 1 << 20
# far apart; the arrays of a call are 1 MB at most
X, W, OFF, OUT, WS = (P(i * 64 * MB) for i in range(1, 6))
M, E, N, K = 512, 2, 64, 96


def _at(p, by):
    return P(p.value + by)


def _off_end(bytes_):
    """Last 16-byte aligned address that still touches an array of that size."""
    return (bytes_ - 1) // 16 * 16


@pytest.mark.parametrize("base,size", [(X, M * K * 2), (W, E * N * K * 2), (OFF, (E + 1) * 4)])
def test_grouped_mm_refuses_an_output_in_an_operand(base, size):
    mm = moeq._load().moeq_grouped_mm
    for by in (0, _off_end(size), -(M * N * 2 - 16)):
        assert mm(X, W, OFF, M, E, N, K, _at(base, by), None) == -1


@pytest.mark.parametrize("base,size", [(X, M * N * 2), (W, E * N * K * 2), (OFF, (E + 1) * 4)])
def test_grad_input_refuses_an_output_in_an_operand(base, size):
    dx = moeq._load().moeq_grouped_mm_grad_input
    for by in (0, _off_end(size), -(M * K * 2 - 16)):
        assert dx(X, W, OFF, M, E, N, K, _at(base, by), None) == -1


@pytest.mark.parametrize("dtype,item", [(1, 2), (2, 4)])
def test_grad_weight_refuses_outputs_and_workspaces_in_operands(dtype, item):
    lib = moeq._load()
    rows = 2048   # long enough for segments
    need = lib.moeq_grouped_mm_grad_weight_workspace_bytes(rows, E, N, K)
    assert need > 0

    def dw(out, ws):
        return lib.moeq_grouped_mm_grad_weight(W, X, OFF, rows, E, N, K, dtype, out, ws, need, None)

    for base, size in ((W, rows * N * 2), (X, rows * K * 2), (OFF, (E + 1) * 4)):
        for by in (0, _off_end(size)):
            assert dw(_at(base, by), WS) == -1
            assert dw(OUT, _at(base, by)) == -1
        assert dw(_at(base, -(E * N * K * item - 16)), WS) == -1
        assert dw(OUT, _at(base, 16 - need)) == -1
    assert dw(OUT, _at(OUT, E * N * K * item - 16)) == -1
    assert dw(_at(WS, _off_end(need)), WS) == -1


def _qw(q, c, e=1, r=M, k=K):
    return moeq._QW(moeq.FMT_MXFP4, e, r, k, 32, q.value, 0, c.value)


def test_mxfp4_calls_refuse_results_in_operands():
    lib = moeq._load()
    x, w = _qw(X, _at(X, 8 * MB)), _qw(W, _at(W, 8 * MB), E, N)
    for q in (x, w):
        rows = q.num_experts * q.rows
        for base, size in ((q.qdata, rows * K // 2), (q.scale_codes, rows * K // 32), (OFF.value, (E + 1) * 4)):
            for by in (0, _off_end(size), -(M * N * 2 - 16)):
                assert lib.moeq_grouped_mm_mxfp4(ctypes.byref(x), ctypes.byref(w), OFF, P(base + by), None) == -1
    for base, size in ((x.qdata, M * K // 2), (x.scale_codes, M * K // 32)):
        for by in (0, _off_end(size), -(M * K * 2 - 16)):
            assert lib.moeq_dequantize_mxfp4(ctypes.byref(x), P(base + by), None) == -1
            # (the input of the quantizer at the same places)
            assert lib.moeq_quantize_mxfp4(P(base + by), ctypes.byref(x), None) == -1
    assert lib.moeq_quantize_mxfp4(OUT, ctypes.byref(_qw(X, _at(X, M * K // 2 - 16))), None) == -1


def test_clipping_refuses_a_norm_or_workspace_in_a_gradient():
    lib = moeq._load()
    need = lib.moeq_clip_grad_norm_workspace_bytes(1)
    src, dst = X.value, W.value

    def clip(norm, ws, s=src, d=dst):
        t = array.array("q", [s, d, 1000, 2])
        return lib.moeq_clip_grad_norm(t.buffer_info()[0], 1, 1.0, P(norm), P(ws), need, None)

    for at in (src, dst, src + 3984, dst + 3984):
        assert clip(at + 12, WS.value) == -1
        assert clip(OUT.value, at) == -1
    assert clip(src + 12, WS.value, d=src) == -1   # in place
    assert clip(WS.value + 8, WS.value) == -1
    assert clip(OUT.value, src + 16 - need) == -1
