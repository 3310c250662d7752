"""GPU: MXFP4 quantize and dequantize against the oracle, bit for bit."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from oracle.mxfp4 import mxfp4_dequantize, mxfp4_quantize
from tests.gpu_common import DEV, dev_bf16, host, host_bits, require_native, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _check(bits):
    q = moeq.moeq_quantize_mxfp4(dev_bf16(bits))
    codes, scales = mxfp4_quantize(bits)
    shape = codes.shape if codes.ndim == 3 else (1, *codes.shape)
    assert q.scales is None and q.blocksize == 32
    assert np.array_equal(host(q.scale_codes), scales.reshape(*shape[:2], -1))
    assert np.array_equal(host(q.qdata), codes.reshape(shape))
    back = host(moeq.moeq_dequantize(q).float()).astype(np.float64)
    want = mxfp4_dequantize(codes, scales).reshape(back.shape)
    assert np.array_equal(back, want, equal_nan=True)   # every value is a bf16
    return q


@pytest.mark.parametrize("shape", [(1, 1, 32), (1, 3, 96), (5, 7, 160), (2, 64, 2880), (3, 33, 8192), (1, 1, 65536)])
def test_random_tensors(shape):
    say(f"mxfp4 {shape}")
    rng = np.random.default_rng(11)
    w = rng.standard_normal(shape) * np.exp2(rng.integers(-20, 20, (*shape[:2], 1)))
    _check(host_bits(torch.from_numpy(w).to(torch.bfloat16)))


def test_every_bf16_against_every_block_scale():
    # each finite bf16 magnitude pattern as a value of blocks whose largest
    # magnitude is in any binade above it, or itself
    say("mxfp4 exhaustive")
    top = np.arange(0, 255, dtype=np.uint32)[:, None] << 7 | 0x7f     # largest of each binade
    vals = np.concatenate([np.arange(0x7f80, dtype=np.uint32)] * 2)
    vals[0x7f80:] |= 0x8000
    per = 31
    pad = -len(vals) % per
    vals = np.concatenate([vals, np.zeros(pad, np.uint32)]).reshape(-1, per)
    for lo in range(0, 255, 51):
        t = top[lo:lo + 51]
        v = np.where((vals & 0x7fff)[None] <= t[:, :, None], vals[None], 0)
        rows = np.concatenate([np.broadcast_to(t[:, :, None], (*v.shape[:2], 1)), v], -1)
        _check(rows.reshape(rows.shape[0], -1).astype(np.uint16))


def test_special_blocks():
    say("mxfp4 special")
    bits = np.zeros((4, 64), np.uint16)
    bits[0, 5], bits[1, 40], bits[2, 0], bits[2, 63] = 0x7f80, 0x7fc1, 0xff80, 0xffc0   # inf, nan, -inf, -nan
    bits[:, 20] = 0x3f80
    bits[3, :] = 0x8000                                                               # -0
    q = _check(bits)
    assert host(q.scale_codes)[0].tolist() == [[255, 0], [125, 255], [255, 255], [0, 0]]


def test_every_scale_byte_reads_back():
    say("mxfp4 scales")
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1)).reshape(256, 256)       # every pair of codes
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    q = moeq.QWeight(moeq.FMT_MXFP4, 1, 256, 512, torch.from_numpy(codes[None]).to(DEV), None,
                     torch.from_numpy(scales[None]).to(DEV))
    got = host(moeq.moeq_dequantize(q).float())[0]
    with np.errstate(over="ignore"):
        want = host(torch.from_numpy(mxfp4_dequantize(codes, scales)).to(torch.float32).to(torch.bfloat16).float())
    assert np.array_equal(got, want, equal_nan=True)


def test_out_buffers_streams_and_empty():
    say("mxfp4 out / stream")
    w = torch.randn(2, 8, 64, device=DEV).to(torch.bfloat16)
    ref = moeq.moeq_quantize_mxfp4(w)
    q = moeq.QWeight.empty(moeq.FMT_MXFP4, 2, 8, 64, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert moeq.moeq_quantize_mxfp4(w, out=q, stream=s) is q
    back = moeq.moeq_dequantize(q, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(q.qdata, ref.qdata) and torch.equal(q.scale_codes, ref.scale_codes)
    assert torch.equal(back, moeq.moeq_dequantize(ref))
    assert torch.equal(moeq.moeq_dequantize(ref.expert(1)), back[1:])
    e = moeq.moeq_quantize_mxfp4(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    assert e.shape == (1, 0, 64) and moeq.moeq_dequantize(e).shape == (1, 0, 64)
