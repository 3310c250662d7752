"""Refusals of the MXFP4, grouped-product and clipping entry points, on the
host: the binding's structural checks on CPU tensors, and the library's own
before any HIP call."""

import array
import ctypes
import os

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq

pytestmark = pytest.mark.skipif(not os.path.exists(moeq.library_path()), reason="libmoeq.so not built")

P = ctypes.c_void_p
BF = torch.bfloat16


def _mx(E=2, R=8, C=64):
    return moeq.QWeight.empty(moeq.FMT_MXFP4, E, R, C, device="cpu")


def _off(E=2):
    return torch.zeros(E + 1, dtype=torch.int32)


def test_mxfp4_layout():
    q = _mx()
    assert q.scales is None and q.blocksize == 32
    assert [s for _, s, _ in q.layout()] == [(2, 8, 32), (2, 8, 2)]
    q.validate_layout()
    assert q.nbytes() == 2 * 8 * (32 + 2)
    assert q.expert(1).validate_layout().shape == (1, 8, 64)
    assert q.like("cpu").validate_layout().scales is None
    q.scales = torch.empty((2, 16))
    with pytest.raises(ValueError):
        q.validate_layout()
    q = _mx()
    q.scale_codes = q.scale_codes[:, :-1].contiguous()
    with pytest.raises(ValueError):
        q.validate_layout()
    with pytest.raises(ValueError):
        _mx(C=48).validate_layout()


def test_mxfp4_calls_refuse():
    w = torch.empty((2, 8, 64), dtype=BF)
    with pytest.raises(ValueError):
        moeq.moeq_quantize_mxfp4(torch.empty((2, 8, 48), dtype=BF))
    with pytest.raises(ValueError):
        moeq.moeq_quantize_mxfp4(torch.empty(64, dtype=BF))
    with pytest.raises(TypeError):
        moeq.moeq_quantize_mxfp4(w.float())
    with pytest.raises(ValueError):
        moeq.moeq_quantize_mxfp4(w, out=_mx(R=4))
    with pytest.raises(ValueError):
        moeq.moeq_quantize_mxfp4(w, out=moeq.QWeight.empty(moeq.FMT_NF4, 2, 8, 64, device="cpu"))
    with pytest.raises(ValueError):
        moeq.moeq_quantize_nf4(w, out=_mx())
    with pytest.raises(TypeError):   # everything right but on the CPU
        moeq.moeq_quantize_mxfp4(w, out=_mx())
    with pytest.raises(TypeError):
        moeq.moeq_dequantize(_mx())


def test_grouped_calls_refuse():
    x, w, dy = torch.empty((5, 16), dtype=BF), torch.empty((2, 24, 16), dtype=BF), torch.empty((5, 24), dtype=BF)
    bad = [
        (ValueError, moeq.moeq_grouped_mm, (x[:, :8].contiguous(), w, _off()), {}),
        (ValueError, moeq.moeq_grouped_mm, (x, w, _off(3)), {}),
        (TypeError, moeq.moeq_grouped_mm, (x, w, _off().long()), {}),
        (TypeError, moeq.moeq_grouped_mm, (x.float(), w, _off()), {}),
        (ValueError, moeq.moeq_grouped_mm, (x, w.transpose(1, 2), _off()), {}),
        (ValueError, moeq.moeq_grouped_mm, (x, w[0], _off()), {}),
        (ValueError, moeq.moeq_grouped_mm, (x, w, _off()), dict(out=torch.empty((5, 16), dtype=BF))),
        (ValueError, moeq.moeq_grouped_mm_grad_input, (x, w, _off()), {}),
        (ValueError, moeq.moeq_grouped_mm_grad_input, (dy, w, _off()), dict(grad_x=torch.empty((4, 16), dtype=BF))),
        (ValueError, moeq.moeq_grouped_mm_grad_weight, (dy, x[:4], _off()), {}),
        (TypeError, moeq.moeq_grouped_mm_grad_weight, (dy, x, _off()), dict(dtype=torch.float16)),
        (ValueError, moeq.moeq_grouped_mm_grad_weight, (dy, x, _off()), dict(grad_w=torch.empty((2, 16, 24)))),
        (ValueError, moeq.moeq_grouped_mm_grad_weight, (dy, x, _off()[:1]), {}),
        (ValueError, moeq.moeq_grouped_mm_mxfp4, (_mx(), _mx(), _off()), {}),                # x must be one "expert"
        (ValueError, moeq.moeq_grouped_mm_mxfp4, (_mx(1, 5, 32), _mx(), _off()), {}),        # columns differ
        (ValueError, moeq.moeq_grouped_mm_mxfp4, (_mx(1), moeq.QWeight.empty(moeq.FMT_NF4, 2, 8, 64, "cpu"), _off()), {}),
        (TypeError, moeq.moeq_grouped_mm_mxfp4, (x, _mx(), _off()), {}),
        (ValueError, moeq.moeq_grouped_mm_mxfp4, (_mx(1), _mx(), _off(3)), {}),
        # everything right but on the CPU
        (TypeError, moeq.moeq_grouped_mm, (x, w, _off()), {}),
        (TypeError, moeq.moeq_grouped_mm_grad_input, (dy, w, _off()), {}),
        (TypeError, moeq.moeq_grouped_mm_grad_weight, (dy, x, _off()), {}),
        (TypeError, moeq.moeq_grouped_mm_mxfp4, (_mx(1), _mx(), _off()), {}),
    ]
    for err, fn, args, kw in bad:
        with pytest.raises(err):
            fn(*args, **kw)


def test_clip_refuses():
    g = [torch.zeros(4), torch.zeros(3, dtype=BF)]
    bad = [
        (ValueError, [], {}),
        (TypeError, [torch.zeros(4, dtype=torch.float16)], {}),
        (TypeError, [None], {}),
        (ValueError, [torch.zeros((4, 4)).t()[:2]], {}),
        (ValueError, g, dict(out=[torch.zeros(4)])),
        (TypeError, g, dict(out=[torch.zeros(4), torch.zeros(3)])),
        (ValueError, g, dict(out=[torch.zeros(5), torch.zeros(3, dtype=BF)])),
        (TypeError, g, {}),   # on the CPU
    ]
    for err, grads, kw in bad:
        with pytest.raises(err):
            moeq.moeq_clip_grad_norm(grads, 1.0, **kw)


def _qw(fmt=4, E=1, R=4, C=64, bs=32, q=256, s=0, c=1024):
    return moeq._QW(fmt, E, R, C, bs, q, s, c)


def test_library_refuses_mxfp4_before_any_device_call():
    lib = moeq._load()

    def quant(q, w=4096):
        return lib.moeq_quantize_mxfp4(P(w), ctypes.byref(q), None)

    assert quant(_qw(fmt=1)) == -4
    assert quant(_qw(C=48)) == -3
    assert quant(_qw(bs=64)) == -3
    assert quant(_qw(c=0)) == -1
    assert quant(_qw(s=512)) == -1        # the format has no fp32 scales
    assert quant(_qw(R=0)) == -1
    assert quant(_qw(q=8)) == -5
    assert quant(_qw(c=1032)) == -5
    assert quant(_qw(), w=0) == -1
    assert quant(_qw(), w=4098) == -5
    assert lib.moeq_quantize_mxfp4(P(4096), None, None) == -1
    assert lib.moeq_dequantize_mxfp4(ctypes.byref(_qw()), P(0), None) == -1
    assert lib.moeq_dequantize_mxfp4(ctypes.byref(_qw()), P(8), None) == -5
    # the calls of the other formats keep refusing it
    assert lib.moeq_quantize_nf4(P(4096), ctypes.byref(_qw()), None) == -4
    assert lib.moeq_dequantize(ctypes.byref(_qw()), P(4096), None) == -4
    assert lib.moeq_qweight_copy_async(ctypes.byref(_qw()), ctypes.byref(_qw()), None) == -4
    gu, dn = _qw(R=128, C=64), _qw(R=64, C=64)
    assert lib.moeq_experts_forward(P(4096), P(4096), P(4096), 2, 1, ctypes.byref(gu), ctypes.byref(dn), P(4096),
                                    P(4096), 1 << 30, None) == -4


def test_library_refuses_grouped_before_any_device_call():
    lib = moeq._load()

    def mm(M=4, E=2, N=16, K=24, x=4096, w=4096, off=4096, out=4096):
        return lib.moeq_grouped_mm(P(x), P(w), P(off), M, E, N, K, P(out), None)

    assert mm(M=-1) == -1 and mm(E=0) == -1 and mm(N=0) == -1 and mm(K=0) == -1
    assert mm(N=12) == -2 and mm(K=20) == -2 and mm(E=1025) == -2
    assert mm(N=1 << 21) == -2 and mm(M=(1 << 28) + 1) == -2
    assert mm(N=1 << 20, K=1 << 10) == -2          # N*K*2 = 2^31
    assert mm(M=1 << 28, N=1 << 16) == -2          # too many tiles
    assert mm(x=0) == -1 and mm(w=0) == -1 and mm(off=0) == -1 and mm(out=0) == -1
    assert mm(x=4104) == -5 and mm(w=4104) == -5 and mm(out=4104) == -5
    assert mm(M=0, x=0, out=0) == 0                 # no rows: a valid no-op

    def dx(M=4, E=2, N=16, K=24, dy=4096):
        return lib.moeq_grouped_mm_grad_input(P(dy), P(4096), P(4096), M, E, N, K, P(4096), None)

    assert dx(N=12) == -2 and dx(dy=0) == -1 and dx(dy=4104) == -5 and dx(M=0) == 0
    assert dx(M=1 << 28, K=1 << 16) == -2

    def dw(M=4, E=2, N=16, K=24, dtype=2, out=4096, x=4096, ws=0, nbytes=0):
        return lib.moeq_grouped_mm_grad_weight(P(4096), P(x), P(4096), M, E, N, K, dtype, P(out), P(ws), nbytes, None)

    need = lib.moeq_grouped_mm_grad_weight_workspace_bytes
    assert need(4, 2, 16, 24) == 0 and need(1 << 20, 2, 16, 24) > 0 and need(1 << 20, 2, 16, 20) == 0
    assert dw(M=1 << 20) == -6 and dw(M=1 << 20, ws=4096, nbytes=64) == -6
    assert dw(M=1 << 20, ws=4100, nbytes=need(1 << 20, 2, 16, 24)) == -5

    assert dw(dtype=3) == -4 and dw(out=0) == -1 and dw(out=4104) == -5 and dw(K=20) == -2 and dw(x=0) == -1

    def mx(x, w, off=4096, out=4096):
        return lib.moeq_grouped_mm_mxfp4(ctypes.byref(x), ctypes.byref(w), P(off), P(out), None)

    w = _qw(E=3, R=16)
    assert mx(_qw(E=2), w) == -2 and mx(_qw(C=32), w) == -2 and mx(_qw(), _qw(R=12)) == -2
    assert mx(_qw(fmt=1, bs=64, s=512, c=0), w) == -4
    assert mx(_qw(), w, off=0) == -1 and mx(_qw(), w, out=0) == -1 and mx(_qw(), w, out=4104) == -5


def test_library_refuses_clipping_before_any_device_call():
    lib = moeq._load()
    need = lib.moeq_clip_grad_norm_workspace_bytes(2)
    assert need > 0 and lib.moeq_clip_grad_norm_workspace_bytes(-1) == 0
    assert lib.moeq_clip_grad_norm_workspace_bytes(1000) > need

    def clip(rows, max_norm=1.0, norm=64, ws=4096, nbytes=need, count=None):
        t = array.array("q", [v for r in rows for v in r])
        return lib.moeq_clip_grad_norm(t.buffer_info()[0] if rows else None, len(rows) if count is None else count,
                                       max_norm, P(norm), P(ws), nbytes, None)

    ok = (1 << 20, 1 << 20, 100, 2)
    assert clip([ok], count=-1) == -1 and clip([], count=1) == -1
    assert clip([ok], max_norm=-1.0) == -1 and clip([ok], max_norm=float("nan")) == -1
    assert clip([ok], norm=0) == -1 and clip([ok], norm=66) == -5
    assert clip([(0, 4096, 4, 2)]) == -1 and clip([(4096, 0, 4, 2)]) == -1 and clip([(4096, 4096, -1, 2)]) == -1
    assert clip([(4096, 4096, 4, 3)]) == -4
    assert clip([(4098, 4098, 4, 2)]) == -5 and clip([(4097, 4097, 4, 1)]) == -5
    assert clip([ok], ws=0) == -6 and clip([ok], nbytes=8) == -6 and clip([ok], ws=4100) == -5
    two = (1 << 20) + 200
    assert clip([ok, (two, two, 10, 1)]) == -1                       # overlapping, both in place
    assert clip([ok, (1 << 21, two, 10, 1)]) == -1                   # a destination inside another tensor
    assert clip([(1 << 20, 1 << 22, 100, 2), (1 << 21, (1 << 22) + 396, 10, 2)]) == -1   # two destinations
