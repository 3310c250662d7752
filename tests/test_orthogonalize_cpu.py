"""Refusals of the orthogonalised update, on the host: the binding's checks on
CPU tensors, and the library's own before any HIP call."""

import array
import ctypes
import os

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq

pytestmark = pytest.mark.skipif(not os.path.exists(moeq.library_path()), reason="libmoeq.so not built")
P = ctypes.c_void_p
FAR = 1 << 40


def test_binding_refuses():
    g, f = torch.zeros((2, 4, 6)), moeq.moeq_orthogonalize
    bad = [
        (ValueError, (g[0, 0],), {}),
        (ValueError, (g[None],), {}),
        (ValueError, (g.transpose(1, 2),), {}),
        (TypeError, (g.half(),), {}),
        (TypeError, (g.double(),), {}),
        (ValueError, (g,), dict(steps=0)),
        (ValueError, (g,), dict(coefficients=(1.0, 2.0))),
        (ValueError, (g,), dict(coefficients=[(1.0, 2.0, 3.0)] * 4)),
        (ValueError, (g,), dict(coefficients=())),
        (ValueError, (g,), dict(out=torch.zeros((2, 6, 4), dtype=torch.bfloat16))),
        (TypeError, (g,), dict(out=torch.zeros((2, 4, 6)))),
        (TypeError, (g,), {}),   # on the CPU
    ]
    for err, args, kw in bad:
        with pytest.raises(err):
            f(*args, **kw)


def _call(g=FAR, dtype=2, E=2, N=8, K=24, table=(1.0, 2.0, 3.0), steps=1, out=2 * FAR, ws=3 * FAR, nbytes=1 << 40):
    t = array.array("f", table)
    return moeq._load().moeq_orthogonalize(P(g), dtype, E, N, K, t.buffer_info()[0] if table else None, steps, P(out), P(ws),
                                           nbytes, None)


def test_library_refuses():
    assert _call(E=0) == -1 and _call(N=0) == -1 and _call(K=-1) == -1 and _call(g=0) == -1 and _call(out=0) == -1
    assert _call(table=()) == -1 and _call(steps=0) == -1 and _call(table=(1.0,) * 195, steps=65) == -1
    assert _call(table=(1.0, float("nan"), 0.0)) == -1 and _call(table=(1.0, 1.0, 1.0, float("inf"), 1.0, 1.0), steps=2) == -1
    assert _call(dtype=3) == -4 and _call(dtype=0) == -4
    assert _call(N=(1 << 20) + 1) == -2 and _call(N=40000, K=40000) == -2 and _call(E=65536) == -2
    assert _call(E=64, N=8, K=1 << 20) == -2 and _call(E=16, N=1 << 15, K=1 << 15) == -2
    assert _call(g=FAR + 2) == -5 and _call(g=FAR + 1, dtype=1) == -5 and _call(out=2 * FAR + 8) == -5 and _call(ws=3 * FAR + 8) == -5
    need = moeq.moeq_orthogonalize_workspace_bytes(2, 8, 24)
    assert need > 0 and _call(ws=0) == -6 and _call(nbytes=need - 1) == -6
    assert moeq.moeq_orthogonalize_workspace_bytes(2, 0, 24) == 0 and moeq.moeq_orthogonalize_workspace_bytes(1, 40000, 40000) == 0
    assert _call(out=FAR) == -1 and _call(out=FAR + 2 * 8 * 24 * 4 - 16) == -1 and _call(out=3 * FAR) == -1 and _call(ws=FAR) == -1
