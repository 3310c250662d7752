"""Refusals of the feed-forward block's entry points, on the host: the
binding's structural checks on CPU tensors, and the library's own before any
HIP call."""

import ctypes
import os

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq

pytestmark = pytest.mark.skipif(not os.path.exists(moeq.library_path()), reason="libmoeq.so not built")
P = ctypes.c_void_p
BF = torch.bfloat16


def _t(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype)


def test_binding_refuses():
    x, w1, w2, off, gu = _t(5, 16), _t(2, 48, 16), _t(2, 16, 24), torch.zeros(3, dtype=torch.int32), _t(5, 48, dtype=torch.float32)
    f, b = moeq.moeq_grouped_ffn, moeq.moeq_grouped_ffn_backward
    bad = [
        (ValueError, f, (x[0], w1, w2, off), {}),
        (ValueError, f, (_t(5, 8), w1, w2, off), {}),
        (ValueError, f, (x, _t(2, 40, 16), w2, off), {}),
        (ValueError, f, (x, _t(3, 48, 16), w2, off), {}),
        (ValueError, f, (x, w1[0], w2, off), {}),
        (ValueError, f, (x, w1, w2.transpose(1, 2), off), {}),
        (ValueError, f, (x, w1, w2, off[:2]), {}),
        (TypeError, f, (x, w1, w2, off.long()), {}),
        (TypeError, f, (x.float(), w1, w2, off), {}),
        (TypeError, f, (x, w1.half(), w2, off), {}),
        (ValueError, f, (x, w1, w2, off), dict(out=_t(4, 16))),
        (ValueError, f, (x, w1, w2, off), dict(gu=_t(5, 24, dtype=torch.float32))),
        (TypeError, f, (x, w1, w2, off), dict(gu=_t(5, 48))),
        (ValueError, b, (_t(4, 16), x, w1, w2, off, gu), {}),
        (ValueError, b, (x, x, w1, w2, off, _t(5, 24)), {}),
        (TypeError, b, (x, x, w1, w2, off, gu), dict(dtype=torch.float16)),
        (TypeError, b, (x, x, w1, w2, off, gu), dict(grad_gate_up=_t(2, 48, 16), grad_down=_t(2, 16, 24, dtype=torch.float32))),
        (ValueError, b, (x, x, w1, w2, off, gu), dict(grad_down=_t(2, 24, 16))),
        (ValueError, b, (x, x, w1, w2, off, gu), dict(grad_x=_t(5, 24))),
        # everything right but on the CPU
        (TypeError, f, (x, w1, w2, off), {}),
        (TypeError, b, (x, x, w1, w2, off, gu), {}),
    ]
    for err, fn, args, kw in bad:
        with pytest.raises(err):
            fn(*args, **kw)


FAR = 1 << 40


def _forward(M=4, E=2, H=16, I=24, x=FAR, w1=2 * FAR, w2=3 * FAR, off=4 * FAR, gu=0, out=5 * FAR, ws=6 * FAR, nbytes=1 << 40):
    return moeq._load().moeq_grouped_ffn(P(x), P(w1), P(w2), P(off), M, E, H, I, P(gu), P(out), P(ws), nbytes, None)


def _backward(M=4, E=2, H=16, I=24, dtype=2, dy=FAR, x=2 * FAR, w1=3 * FAR, w2=4 * FAR, off=5 * FAR, gu=6 * FAR, dx=7 * FAR,
              dw1=8 * FAR, dw2=9 * FAR, ws=10 * FAR, nbytes=1 << 40):
    return moeq._load().moeq_grouped_ffn_backward(P(dy), P(x), P(w1), P(w2), P(off), P(gu), M, E, H, I, dtype, P(dx), P(dw1),
                                                  P(dw2), P(ws), nbytes, None)


def test_library_refuses_sizes():
    for call in (_forward, _backward):
        assert call(M=-1) == -1 and call(E=0) == -1 and call(H=0) == -1 and call(I=0) == -1 and call(I=-8) == -1
        assert call(H=12) == -2 and call(I=12) == -2 and call(E=1025) == -2 and call(M=(1 << 28) + 8) == -2
        assert call(I=1 << 20) == -2 and call(I=2 ** 31 - 8) == -2 and call(H=1 << 21) == -2
        assert call(H=1 << 15, I=1 << 14) == -2                # 2I * H * 2 = 2^31
        assert call(M=1 << 28, H=1 << 16) == -2                # too many tiles
    need = moeq.moeq_grouped_ffn_workspace_bytes
    assert need(4, 2, 16, 24) == 4 * 24 * 2 and need(4, 2, 16, 20) == 0 and need(0, 2, 16, 24) == 0
    back = moeq.moeq_grouped_ffn_backward_workspace_bytes
    sums = moeq.moeq_grouped_mm_grad_weight_workspace_bytes
    assert back(4, 2, 16, 24) == 4 * 24 * 6 and back(4, 2, 12, 24) == 0
    M = 1 << 20
    assert back(M, 2, 16, 24) == M * 24 * 6 + max(sums(M, 2, 48, 16), sums(M, 2, 16, 24))


def test_library_refuses_pointers_and_workspaces():
    for k in ("x", "w1", "w2", "off", "out"):
        assert _forward(**{k: 0}) == -1, k
    for k in ("x", "w1", "w2", "gu", "out"):
        assert _forward(**{k: FAR * 20 + 8}) == -5, k
    assert _forward(ws=0) == -6 and _forward(nbytes=4 * 24 * 2 - 1) == -6 and _forward(ws=6 * FAR + 4) == -5
    assert _forward(M=0, x=0, w1=0, w2=0, off=0, out=0, ws=0, nbytes=0) == 0   # a valid no-op
    for k in ("dy", "x", "w1", "w2", "off", "gu", "dx", "dw1", "dw2"):
        assert _backward(**{k: 0}) == -1, k
    for k in ("dy", "x", "w1", "w2", "gu", "dx", "dw1", "dw2"):
        assert _backward(**{k: FAR * 20 + 8}) == -5, k
    assert _backward(dtype=3) == -4
    assert _backward(ws=0) == -6 and _backward(nbytes=4 * 24 * 6 - 1) == -6 and _backward(ws=10 * FAR + 4) == -5
    assert _backward(M=0, dw1=0) == -1 and _backward(M=0, off=0) == -1


def test_library_refuses_overlaps():
    assert _forward(out=FAR) == -1                       # x itself
    assert _forward(out=FAR + 4 * 16 * 2 - 16) == -1     # its last row
    assert _forward(out=2 * FAR) == -1 and _forward(out=3 * FAR) == -1 and _forward(out=4 * FAR) == -1
    assert _forward(ws=FAR) == -1 and _forward(ws=5 * FAR) == -1 and _forward(gu=6 * FAR) == -1 and _forward(gu=5 * FAR) == -1
    outs = dict(dx=7 * FAR, dw1=8 * FAR, dw2=9 * FAR, ws=10 * FAR)
    for k in outs:
        for at in range(1, 7):
            assert _backward(**{k: at * FAR}) == -1, (k, at)
        for j, at in outs.items():
            if j != k:
                assert _backward(**{k: at}) == -1, (k, j)
