"""GPU: the operators of trained experts as they are used together (route, block,
gradients, clipping, orthogonalised update, then serving in FP8), each stage held
to its own bound on the inputs that it got; arrays past 32-bit offsets; calls on
two streams at once."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from tests.gpu_common import DEV, host, require_native, say
from tests.test_gpu_ffn import _check_backward, _check_forward
from tests.test_gpu_fp8 import _check_product, _check_quantize
from tests.test_gpu_grouped import _f64
from tests.test_gpu_orthogonalize import _check as _check_orthogonal

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _step(x, gate, w1, w2, target, K, served):
    """One training step of the experts and the next forward pass in FP8."""
    idx, wts, r = moeq.moeq_router_route(x, gate, K, renormalize=True)
    token = (r.perm // K).long()
    rows, weight = x[token], wts.flatten()[r.perm.long()]
    out, gu = moeq.moeq_grouped_ffn(rows, w1, w2, r.offsets, save=True)
    y = torch.zeros(x.shape, dtype=F32, device=DEV).index_add_(0, token, out.float() * weight[:, None])
    dy = ((y - target)[token] * weight[:, None]).to(BF16)
    dx, dw1, dw2 = moeq.moeq_grouped_ffn_backward(dy, rows, w1, w2, r.offsets, gu)
    raw = (dw1.clone(), dw2.clone())
    norm = moeq.moeq_clip_grad_norm([dw1, dw2], 1.0)
    o1, o2 = moeq.moeq_orthogonalize(dw1), moeq.moeq_orthogonalize(dw2)
    n1, n2 = (w1 - 0.02 * o1).to(BF16), (w2 - 0.02 * o2).to(BF16)
    q1, q2 = moeq.moeq_quantize_fp8(n1), moeq.moeq_quantize_fp8(n2)
    xq = moeq.moeq_quantize_fp8(rows, moeq.FMT_FP8_ROW)
    gu8 = moeq.moeq_grouped_mm_fp8(xq, q1, r.offsets)
    g, u = gu8.float().chunk(2, 1)
    hq = moeq.moeq_quantize_fp8((torch.nn.functional.silu(g) * u).to(BF16), moeq.FMT_FP8_ROW)
    y8 = moeq.moeq_grouped_mm_fp8(hq, q2, r.offsets)
    if served is not None:
        served.update(locals())
    return y8, n1, n2, norm, dx


def _inputs(T, H, I, E, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    return (r(T, H).to(BF16), (r(E, H) * 0.05).to(BF16), (r(E, 2 * I, H) * H ** -0.5).to(BF16),
            (r(E, H, I) * I ** -0.5).to(BF16), r(T, H))


@pytest.mark.parametrize("T,H,I,E,K", [(1, 64, 16, 8, 2), (200, 192, 144, 8, 2), (600, 128, 48, 33, 4)])
def test_a_step_and_serving(T, H, I, E, K):
    say(f"training step T={T} H={H} I={I} E={E}")
    x, gate, w1, w2, target = _inputs(T, H, I, E, 1)
    s = {}
    _step(x, gate, w1, w2, target, K, s)
    off = host(s["r"].offsets)
    _check_forward(s["rows"], w1, w2, off, s["out"], s["gu"])
    _check_backward(s["dy"], s["rows"], w1, w2, off, s["gu"], (s["dx"], *s["raw"]), 2.0 ** -24)
    total = np.sqrt(sum((_f64(t) ** 2).sum() for t in s["raw"]))
    # the sum and the root are fp64, the norm and the factor one fp32 rounding each, the product another
    assert abs(float(s["norm"]) - total) <= 2.0 ** -23 * total
    for raw, dw in zip(s["raw"], (s["dw1"], s["dw2"])):
        assert np.all(np.abs(_f64(dw) - _f64(raw) * min(1.0, 1.0 / total)) <= 2.0 ** -22 * np.abs(_f64(raw)) + 1e-38)
    for dw, o in ((s["dw1"], s["o1"]), (s["dw2"], s["o2"])):
        pick = [int(np.argmax(np.diff(off))), int(np.argmin(np.diff(off)))]
        _check_orthogonal(dw[pick], o[pick])
    _check_quantize(s["n1"], "tile")
    _check_quantize(s["rows"][None], "row")
    _check_product(s["gu8"], s["xq"], s["q1"], off)
    _check_product(s["y8"], s["hq"], s["q2"], off)


def test_a_captured_step():
    """Captured, and replayed with eager steps and synchronizations between the replays."""
    say("training step captured")
    x, gate, w1, w2, target = _inputs(150, 128, 80, 8, 2)
    _step(x, gate, w1, w2, target, 2, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(x, gate, w1, w2, target, 2, None)
    for k in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device=DEV).manual_seed(k), device=DEV))
        want = [t.clone() for t in _step(x, gate, w1, w2, target, 2, None)]
        graph.replay()
        torch.cuda.synchronize()
        # (two terms a token: index_add_'s order makes no difference)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_two_streams_at_once():
    say("two streams at once")
    x, _, w1, w2, target = _inputs(500, 256, 136, 4, 3)
    off = torch.tensor([0, 100, 100, 260, 500], dtype=torch.int32, device=DEV)
    g = torch.randn((6, 130, 300), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    q = moeq.moeq_quantize_fp8(w1)

    def work(s=None):
        y, gu = moeq.moeq_grouped_ffn(x, w1, w2, off, save=True, stream=s)
        grads = moeq.moeq_grouped_ffn_backward(y, x, w1, w2, off, gu, stream=s)
        z = moeq.moeq_grouped_mm_fp8(moeq.moeq_quantize_fp8(x, moeq.FMT_FP8_ROW, stream=s), q, off, stream=s)
        return [y, gu, *grads, z, moeq.moeq_orthogonalize(g, stream=s)]

    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [work(s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for one in got for a, b in zip(one, want))


def test_block_past_32_bit_offsets():
    """g | u of 9.8 GB: the last expert's rows come out as in a call of their own."""
    say("ffn past 32-bit offsets")
    M, H, I = 150_000, 8, 8192
    g = torch.Generator(device=DEV).manual_seed(5)
    x, dy = (torch.randn((M, H), generator=g, device=DEV).to(BF16) for _ in range(2))
    w1 = torch.randn((2, 2 * I, H), generator=g, device=DEV).to(BF16)
    w2 = (torch.randn((2, H, I), generator=g, device=DEV) * I ** -0.5).to(BF16)
    off = torch.tensor([0, M - 300, M], dtype=torch.int32, device=DEV)
    y, gu = moeq.moeq_grouped_ffn(x, w1, w2, off, save=True)
    dx, dw1, dw2 = moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, off, gu)
    own = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    tail = [t[-300:].contiguous() for t in (x, dy)]
    y1, gu1 = moeq.moeq_grouped_ffn(tail[0], w1[1:].contiguous(), w2[1:].contiguous(), own, save=True)
    d1 = moeq.moeq_grouped_ffn_backward(tail[1], tail[0], w1[1:].contiguous(), w2[1:].contiguous(), own, gu1)
    assert torch.equal(y[-300:], y1) and torch.equal(gu[-300:], gu1)
    assert torch.equal(dx[-300:], d1[0]) and torch.equal(dw1[1], d1[1][0]) and torch.equal(dw2[1], d1[2][0])


def test_fp8_past_32_bit_offsets():
    """Rows of 2.5 GB of codes and weights of 2.7 GB: the last ones as alone."""
    say("fp8 past 32-bit offsets")
    g = torch.Generator(device=DEV).manual_seed(6)
    M, K, E, N = 300_000, 8208, 41, 8192
    x = torch.randn((M, K), generator=g, device=DEV, dtype=BF16)
    xq = moeq.moeq_quantize_fp8(x, moeq.FMT_FP8_ROW)
    tail = moeq.moeq_quantize_fp8(x[-300:].contiguous(), moeq.FMT_FP8_ROW)
    assert torch.equal(xq.qdata[0, -300:].view(torch.uint8), tail.qdata[0].view(torch.uint8))
    assert torch.equal(xq.scales[0, -300:], tail.scales[0])
    assert torch.equal(moeq.moeq_dequantize(xq)[0, -300:], moeq.moeq_dequantize(tail)[0])
    del x
    w = torch.randn((E, N, K), generator=g, device=DEV, dtype=BF16)
    wq, last = moeq.moeq_quantize_fp8(w), moeq.moeq_quantize_fp8(w[-1:].contiguous())
    assert torch.equal(wq.qdata[-1].view(torch.uint8), last.qdata[0].view(torch.uint8)) and torch.equal(wq.scales[-1], last.scales[0])
    assert torch.equal(moeq.moeq_dequantize(wq)[-1], moeq.moeq_dequantize(last)[0])
    del w
    own = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    want = moeq.moeq_grouped_mm_fp8(tail, last, own)
    off = torch.full((E + 1,), 300, dtype=torch.int32, device=DEV)   # only the last expert has rows
    off[:E] = 0
    assert torch.equal(moeq.moeq_grouped_mm_fp8(tail, wq, off), want)
    small = moeq.QWeight(moeq.FMT_FP8_TILE, 1, 16, K, last.qdata[:, :16].contiguous(), last.scales[:, :1].contiguous())
    far = torch.tensor([M - 300, M], dtype=torch.int32, device=DEV)   # only the last rows belong to it
    assert torch.equal(moeq.moeq_grouped_mm_fp8(xq, small, far)[-300:], moeq.moeq_grouped_mm_fp8(tail, small, own))


def test_orthogonalize_past_32_bit_offsets():
    say("orthogonalize past 32-bit offsets")
    g = torch.randn((33, 8192, 8200), generator=torch.Generator(device=DEV).manual_seed(7), device=DEV, dtype=BF16)
    out = moeq.moeq_orthogonalize(g)
    for e in (0, 32):
        assert torch.equal(out[e], moeq.moeq_orthogonalize(g[e]))
