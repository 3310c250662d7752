"""GPU: outputs and workspaces of the grouped products, the MXFP4 format and
the gradient clipping between guard bytes that must come back untouched, with
no rows behind the last expert: a store past the last row, column, expert or
block would otherwise go unseen."""

import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from tests.gpu_common import require_native, say
from tests.test_gpu_guarded import Guarded

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8

ROWS = {
    "one row": [1],
    "few rows": [2, 0, 9, 1, 17, 0, 3, 8],
    "tile borders": [32, 64, 65, 128, 129, 192, 193, 256, 257],
    "long expert": [40] * 20 + [1500],
    "many experts": [(i * 7) % 40 + 1 for i in range(300)],
}


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("N,K", [(8, 8), (16, 264), (264, 16), (72, 136), (520, 1032)])
def test_products(rows, N, K):
    say(f"guarded grouped {rows} N={N} K={K}")
    g = torch.Generator(device="cuda").manual_seed(1)
    sizes = torch.tensor([0] + ROWS[rows])
    off = sizes.cumsum(0).to(torch.int32).cuda()
    M, E = int(sizes.sum()), len(sizes) - 1
    x, dy, w = _randn((M, K), g), _randn((M, N), g), _randn((E, N, K), g)
    y, dx = Guarded((M, N), BF16), Guarded((M, K), BF16)
    assert torch.equal(moeq.moeq_grouped_mm(x, w, off, out=y.t), moeq.moeq_grouped_mm(x, w, off))
    y.check("out")
    assert torch.equal(moeq.moeq_grouped_mm_grad_input(dy, w, off, grad_x=dx.t), moeq.moeq_grouped_mm_grad_input(dy, w, off))
    dx.check("grad_x")
    need = moeq.moeq_grouped_mm_grad_weight_workspace_bytes(M, E, N, K)
    for dtype in (F32, BF16):
        dw, ws = Guarded((E, N, K), dtype), Guarded((need,), U8)
        moeq.moeq_grouped_mm_grad_weight(dy, x, off, grad_w=dw.t, workspace=ws.t)
        dw.check(f"grad_w {dtype}")
        ws.check("workspace")
        assert torch.equal(dw.t, moeq.moeq_grouped_mm_grad_weight(dy, x, off, dtype=dtype))


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("N,K", [(8, 32), (72, 160), (520, 1056)])
def test_mxfp4(rows, N, K):
    say(f"guarded mxfp4 {rows} N={N} K={K}")
    g = torch.Generator(device="cuda").manual_seed(2)
    sizes = torch.tensor([0] + ROWS[rows])
    off = sizes.cumsum(0).to(torch.int32).cuda()
    M, E = int(sizes.sum()), len(sizes) - 1
    x, w = _randn((M, K), g), _randn((E, N, K), g)
    quantized = []
    for t, shape in ((x, (1, M, K)), (w, (E, N, K))):
        probe = moeq.QWeight(moeq.FMT_MXFP4, *shape, None, None)
        q, s = (Guarded(want, dtype) for _, want, dtype in probe.layout())
        quantized.append(moeq.QWeight(moeq.FMT_MXFP4, *shape, q.t, None, s.t))
        moeq.moeq_quantize_mxfp4(t, out=quantized[-1])
        q.check("codes")
        s.check("scales")
        ref = moeq.moeq_quantize_mxfp4(t)
        assert torch.equal(q.t, ref.qdata) and torch.equal(s.t, ref.scale_codes)
        back = Guarded(shape, BF16)
        assert torch.equal(moeq.moeq_dequantize(quantized[-1], out=back.t), moeq.moeq_dequantize(ref))
        back.check("read back")
    y = Guarded((M, N), BF16)
    assert torch.equal(moeq.moeq_grouped_mm_mxfp4(*quantized, off, out=y.t), moeq.moeq_grouped_mm_mxfp4(*quantized, off))
    y.check("out")


@pytest.mark.parametrize("lens", [[1], [1, 2, 3, 5, 31, 33, 255, 257, 1023], [16383, 16385, 40001], [8] * 96 + [3] * 97])
def test_clipping(lens):
    say(f"guarded clip {len(lens)}")
    g = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(n, generator=g, device="cuda").to(F32 if i % 2 else BF16) for i, n in enumerate(lens)]
    out = [Guarded((n,), t.dtype) for n, t in zip(lens, grads)]
    ws = Guarded((moeq.moeq_clip_grad_norm_workspace_bytes(len(lens)),), U8)
    norm = moeq.moeq_clip_grad_norm(grads, 0.25, out=[o.t for o in out], workspace=ws.t)
    ws.check("workspace")
    for o in out:
        o.check("out")
    assert torch.equal(moeq.moeq_clip_grad_norm([o.t.copy_(t) for o, t in zip(out, grads)], 0.25, workspace=ws.t), norm)
    ws.check("workspace")
    for o in out:
        o.check("in place")


def test_an_output_that_is_an_operand_is_refused():
    say("guarded in place")
    g = torch.Generator(device="cuda").manual_seed(4)
    off = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    x, w = _randn((40, 64), g), _randn((2, 64, 64), g)
    keep = [x.clone(), w.clone()]
    calls = [lambda: moeq.moeq_grouped_mm(x, w, off, out=x),
             lambda: moeq.moeq_grouped_mm(x, w, off, out=w.view(128, 64)[:40]),
             lambda: moeq.moeq_grouped_mm_grad_input(x, w, off, grad_x=x),
             lambda: moeq.moeq_grouped_mm_grad_weight(w.view(128, 64), w.view(128, 64), off, grad_w=w)]
    for call in calls:
        with pytest.raises(moeq.MoeqError) as e:
            call()
        assert e.value.status == -1
    assert torch.equal(x, keep[0]) and torch.equal(w, keep[1])
