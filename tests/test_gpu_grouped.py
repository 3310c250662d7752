"""GPU: products grouped by expert, in bf16 (forward and gradients) and MXFP4,
against the 64-bit oracle.

Tolerance, per output: the operands' products are exact in fp32 up to the sum,
which is a chain of at most L (the contraction length) fp32 additions, each
off by at most one unit of 2^-23 of the running sum of magnitudes (the matrix
cores may truncate), and the result is rounded once: half a step of its type.
So |got - exact| <= 2^-8 |exact| (bf16; 2^-24 for fp32) + L 2^-23 sum |a b|
(1 + 2^-8), the last factor for the rounding of the accumulated error."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from oracle.grouped import grouped_mm, grouped_mm_grad_input, grouped_mm_grad_weight
from oracle.mxfp4 import mxfp4_dequantize
from tests.gpu_common import DEV, host, require_native, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _offsets(sizes, before=0):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + np.int32(before)


# (rows per expert, rows before the first, rows behind the last)
ROWS = {
    "one row": ([1], 0, 0),
    "one expert": ([37], 0, 0),
    "no rows": ([0, 0, 0], 0, 0),
    "empty experts": ([0, 5, 0, 0, 70, 1, 0], 0, 0),
    "rows outside": ([3, 0, 17], 2, 6),
    "few rows": ([2, 0, 9, 1, 17, 0, 3, 8], 0, 0),
    "tile borders": ([32, 64, 65, 128, 129, 192, 193, 256, 257], 0, 0),
    "large and small": ([700, 1, 0, 33], 0, 1),
    "many experts": ([(i * 7) % 5 for i in range(150)], 1, 3),
    "one row each": ([1, 0, 2] * 60, 0, 0),
}


def _f64(t):
    return host(t.float()).astype(np.float64)


def _case(rows, N, K, seed=0):
    sizes, before, behind = ROWS[rows]
    g = torch.Generator(device=DEV).manual_seed(seed)
    off = _offsets(sizes, before)
    M = int(off[-1]) + behind
    x = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((len(sizes), N, K), generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn((M, N), generator=g, device=DEV).to(torch.bfloat16)
    for t in (x, dy):   # rows of no expert hold anything
        t[:off[0]] = float("nan")
        t[off[-1]:] = float("inf")
    return x, w, dy, off, torch.from_numpy(off).to(DEV)


def _assert_close(got, want, mag, L, half=2.0 ** -8):
    got = _f64(got)
    live = ~np.isnan(want)
    tol = half * np.abs(want) + L * 2.0 ** -23 * mag * (1 + 2.0 ** -8)
    bad = live & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def _untouched(out, off):
    """Rows of no expert keep what was there."""
    return bool((out[:off[0]] == 7).all() and (out[off[-1]:] == 7).all())


def _clean(t, off):
    a = _f64(t)
    a[:off[0]] = 0
    a[off[-1]:] = 0
    return a


SHAPES = [(8, 8), (520, 136), (16, 64), (64, 16), (72, 136), (256, 256), (264, 520), (1000, 1032)]


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("N,K", SHAPES)
def test_forward_and_gradients(rows, N, K):
    say(f"grouped {rows} N={N} K={K}")
    x, w, dy, off, doff = _case(rows, N, K)
    M = x.shape[0]
    xs, dys, ws = _clean(x, off), _clean(dy, off), _f64(w)

    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    assert moeq.moeq_grouped_mm(x, w, doff, out=y) is y
    _assert_close(y, grouped_mm(xs, ws, off), grouped_mm(np.abs(xs), np.abs(ws), off), K)
    assert _untouched(y, off)

    dx = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=DEV)
    moeq.moeq_grouped_mm_grad_input(dy, w, doff, grad_x=dx)
    _assert_close(dx, grouped_mm_grad_input(dys, ws, off), grouped_mm_grad_input(np.abs(dys), np.abs(ws), off), N)
    assert _untouched(dx, off)

    want, mag = grouped_mm_grad_weight(dys, xs, off), grouped_mm_grad_weight(np.abs(dys), np.abs(xs), off)
    L = int(np.diff(off).max())
    dw = moeq.moeq_grouped_mm_grad_weight(dy, x, doff)
    assert dw.dtype == torch.float32
    _assert_close(dw, want, mag, L, 2.0 ** -24)
    dw16 = moeq.moeq_grouped_mm_grad_weight(dy, x, doff, dtype=torch.bfloat16)
    _assert_close(dw16, want, mag, L)
    assert torch.equal(dw16, dw.to(torch.bfloat16))   # one rounding of the same sums
    for e in np.flatnonzero(np.diff(off) == 0):
        assert not dw[e].any()


@pytest.mark.parametrize("N,K", [(16, 264), (264, 16), (264, 264)])
@pytest.mark.parametrize("sizes", [[1500], [0, 513, 1, 512, 2050, 0, 700], [40] * 70 + [1100]])
def test_gradient_of_long_experts_is_summed_in_segments(N, K, sizes):
    """Segments of 512 rows (more for the square tile): partial sums in fp32,
    added in fp32, so the bound of one long sum holds."""
    say(f"grouped segments {N} {K} {len(sizes)}")
    g = torch.Generator(device=DEV).manual_seed(21)
    off = _offsets(sizes, 3)
    M = int(off[-1]) + 2
    x = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn((M, N), generator=g, device=DEV).to(torch.bfloat16)
    for t in (x, dy):
        t[:3], t[-2:] = float("nan"), float("nan")
    doff = torch.from_numpy(off).to(DEV)
    xs, dys = _clean(x, off), _clean(dy, off)
    want, mag = grouped_mm_grad_weight(dys, xs, off), grouped_mm_grad_weight(np.abs(dys), np.abs(xs), off)
    ws = torch.full((moeq.moeq_grouped_mm_grad_weight_workspace_bytes(M, len(sizes), N, K) + 64,), 0xff,
                    dtype=torch.uint8, device=DEV)   # NaNs, where the call does not write
    for dtype, half in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        dw = moeq.moeq_grouped_mm_grad_weight(dy, x, doff, dtype=dtype, workspace=ws)
        _assert_close(dw, want, mag, max(sizes), half)
        assert (ws[-64:] == 0xff).all()
        assert torch.equal(dw, moeq.moeq_grouped_mm_grad_weight(dy, x, doff, dtype=dtype))


def _mx_random(shape, g):
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(120, 134, (*shape[:-1], shape[-1] // 32), generator=g, device=DEV, dtype=torch.uint8)
    return moeq.QWeight(moeq.FMT_MXFP4, *shape, codes, None, scales)


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("N,K", [(8, 32), (16, 96), (72, 128), (256, 256), (520, 544), (264, 544), (64, 2880), (64, 4128)])
def test_mxfp4_forward(rows, N, K):
    say(f"grouped mxfp4 {rows} N={N} K={K}")
    sizes, before, behind = ROWS[rows]
    off = _offsets(sizes, before)
    M = max(int(off[-1]) + behind, 1)
    g = torch.Generator(device=DEV).manual_seed(5)
    x, w = _mx_random((1, M, K), g), _mx_random((len(sizes), N, K), g)
    x.scale_codes[0, :before] = 255      # NaN rows of no expert
    x.scale_codes[0, off[-1]:] = 255
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    assert moeq.moeq_grouped_mm_mxfp4(x, w, torch.from_numpy(off).to(DEV), out=y) is y
    xs, ws = mxfp4_dequantize(host(x.qdata)[0], host(x.scale_codes)[0]), mxfp4_dequantize(host(w.qdata), host(w.scale_codes))
    xs[:before] = 0
    xs[off[-1]:] = 0
    _assert_close(y, grouped_mm(xs, ws, off), grouped_mm(np.abs(xs), np.abs(ws), off), K)
    assert _untouched(y, off)


def test_mxfp4_nan_blocks_reach_their_outputs_alone():
    say("grouped mxfp4 nan")
    g = torch.Generator(device=DEV).manual_seed(6)
    K, N = 352, 24
    x, w = _mx_random((1, 40, K), g), _mx_random((2, N, K), g)
    off = torch.tensor([0, 15, 40], dtype=torch.int32, device=DEV)
    x.scale_codes[0, 4, 10] = 255
    x.scale_codes[0, 39, 0] = 255
    w.scale_codes[1, 5, 3] = 255
    nan = host(torch.isnan(moeq.moeq_grouped_mm_mxfp4(x, w, off)))
    want = np.zeros((40, N), bool)
    want[4], want[39], want[15:, 5] = True, True, True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_values_of_other_experts_stay_out(bad):
    """A row and a weight that are not finite reach only the results they enter."""
    say(f"grouped not finite {bad}")
    x, w, dy, off, doff = _case("tile borders", 72, 136)
    sizes = ROWS["tile borders"][0]
    ref = [moeq.moeq_grouped_mm(x, w, doff), moeq.moeq_grouped_mm_grad_input(dy, w, doff),
           moeq.moeq_grouped_mm_grad_weight(dy, x, doff)]
    p = int(off[4])          # first row of expert 4
    x[p], dy[p + 1] = bad, bad
    w[6] = bad
    got = [moeq.moeq_grouped_mm(x, w, doff), moeq.moeq_grouped_mm_grad_input(dy, w, doff),
           moeq.moeq_grouped_mm_grad_weight(dy, x, doff)]
    rows = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    rows[off[6]:off[7]] = False
    for r, i in ((p, 0), (p + 1, 1)):
        keep = rows.clone()
        keep[r] = False
        assert torch.equal(got[i][keep], ref[i][keep])
        assert not torch.isfinite(got[i][~keep]).any()
    experts = torch.arange(len(sizes), device=DEV) != 4
    assert torch.equal(got[2][experts], ref[2][experts]) and not torch.isfinite(got[2][4]).all()


def test_gradients_against_differences():
    """<dy, f(x + d) - f(x - d)> / 2 = <dx, d>: the product is linear in x and
    in w, so the difference quotient is exact up to the roundings."""
    say("grouped differences")
    g = torch.Generator(device=DEV).manual_seed(9)
    x, w, dy, off, doff = _case("empty experts", 48, 80)
    M = x.shape[0]
    d = (torch.randint(-2, 3, x.shape, generator=g, device=DEV) / 4).to(torch.bfloat16)
    dw_dir = (torch.randint(-2, 3, w.shape, generator=g, device=DEV) / 4).to(torch.bfloat16)
    dys = _f64(dy)
    dx = _f64(moeq.moeq_grouped_mm_grad_input(dy, w, doff))
    dw = _f64(moeq.moeq_grouped_mm_grad_weight(dy, x, doff))
    # f is linear: f(x + d) - f(x - d) = 2 f(d), formed without cancellation
    for num, ana, mag in ((dys * _f64(moeq.moeq_grouped_mm(d, w, doff)), dx * _f64(d), np.abs(dx * _f64(d))),
                          (dys * _f64(moeq.moeq_grouped_mm(x, dw_dir, doff)), dw * _f64(dw_dir), np.abs(dw * _f64(dw_dir)))):
        # each side's terms carry one rounding to bf16 (2^-8) and fp32 sums
        tol = (2.0 ** -8 + 200 * 2.0 ** -23) * (np.abs(num).sum() + mag.sum())
        assert abs(num.sum() - ana.sum()) <= tol
    assert M == off[-1]


def test_same_bits_and_streams():
    say("grouped streams")
    x, w, dy, off, doff = _case("large and small", 264, 520)
    ref = [moeq.moeq_grouped_mm(x, w, doff)[:off[-1]], moeq.moeq_grouped_mm_grad_input(dy, w, doff)[:off[-1]],
           moeq.moeq_grouped_mm_grad_weight(dy, x, doff)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:   # two calls at once
        got.append([moeq.moeq_grouped_mm(x, w, doff, stream=s)[:off[-1]],
                    moeq.moeq_grouped_mm_grad_input(dy, w, doff, stream=s)[:off[-1]],
                    moeq.moeq_grouped_mm_grad_weight(dy, x, doff, stream=s)])
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_a_call_on_another_stream_does_not_take_memory_in_use():
    """Outputs and workspaces of a call on a side stream come from memory that
    work still queued on the current stream cannot be writing."""
    say("grouped side stream memory")
    g = torch.Generator(device=DEV).manual_seed(17)
    off = torch.tensor([0, 700, 1500], dtype=torch.int32, device=DEV)
    x = torch.randn((1500, 512), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((2, 256, 512), generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn((1500, 256), generator=g, device=DEV).to(torch.bfloat16)
    ref = [moeq.moeq_grouped_mm(x, w, off), moeq.moeq_grouped_mm_grad_weight(dy, x, off),
           moeq.moeq_dequantize(moeq.moeq_quantize_mxfp4(x))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.zeros((1 << 28,), device=DEV)
    torch.cuda.synchronize()
    for _ in range(6):
        big.add_(1.0)                                 # keeps the current stream busy (milliseconds)
    late = [torch.empty_like(t) for t in ref]         # written behind that, freed at once
    for t in late:
        t.fill_(5.0)
    del late, t
    q = moeq.moeq_quantize_mxfp4(x, stream=side)
    got = [moeq.moeq_grouped_mm(x, w, off, stream=side), moeq.moeq_grouped_mm_grad_weight(dy, x, off, stream=side),
           moeq.moeq_dequantize(q, stream=side)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_captured_and_replayed():
    say("grouped graph")
    x, w, dy, off, doff = _case("empty experts", 72, 160)
    xq, wq = moeq.moeq_quantize_mxfp4(x), moeq.moeq_quantize_mxfp4(w)

    def step():
        moeq.moeq_quantize_mxfp4(x, out=xq)
        return [moeq.moeq_grouped_mm(x, w, doff), moeq.moeq_grouped_mm_mxfp4(xq, wq, doff),
                moeq.moeq_grouped_mm_grad_input(dy, w, doff), moeq.moeq_grouped_mm_grad_weight(dy, x, doff)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):   # new inputs and new offsets each time, eager work between
        g = torch.Generator(device=DEV).manual_seed(100 + i)
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        dy.copy_(torch.randn(dy.shape, generator=g, device=DEV))
        sizes = np.roll(ROWS["empty experts"][0], i)
        doff.copy_(torch.from_numpy(_offsets(sizes)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
        torch.cuda.synchronize()


def test_routed_chain_matches_the_experts_forward():
    """Router -> sorted rows -> grouped gate/up, SwiGLU, grouped down ->
    weighted sum, with dequantized NF4 experts, against the fused forward:
    both have the same rounding points but for bf16 g and u here."""
    say("grouped chain")
    import moeq_synth as syn
    s = syn.SHAPES["tiny"]
    T = 300
    gu, dn, x, _, _ = syn.layer_inputs(s, T, device=DEV)
    gate = syn.router_weight(s.E, s.H, device=DEV)
    qg, qd = moeq.moeq_quantize_nf4(gu), moeq.moeq_quantize_nf4(dn)
    idx, wts, r = moeq.moeq_router_route(x, gate, s.K)
    ref = moeq.moeq_experts_forward_routed(x, idx, wts, qg, qd, r)
    xs = x[(r.perm // s.K).long()]
    g, u = moeq.moeq_grouped_mm(xs, moeq.moeq_dequantize(qg), r.offsets).float().chunk(2, -1)
    h = (torch.nn.functional.silu(g) * u).to(torch.bfloat16)
    y = moeq.moeq_grouped_mm(h, moeq.moeq_dequantize(qd), r.offsets).float()
    out = (y[r.slot.long()].view(T, s.K, -1) * wts[..., None]).sum(1)
    err = (out - ref.float()).norm() / ref.float().norm()
    assert err <= 8e-3, float(err)   # four bf16 roundings of RMS 2^-8 / sqrt(3) each at most, in quadrature


def test_mxfp4_layer_matches_its_dequantized_weights():
    """Quantize -> grouped product, and the same on the read-back values in bf16."""
    say("grouped mxfp4 layer")
    g = torch.Generator(device=DEV).manual_seed(12)
    off = torch.tensor([0, 100, 100, 260, 301], dtype=torch.int32, device=DEV)
    x = torch.randn((301, 288), generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn((4, 120, 288), generator=g, device=DEV) * 0.02).to(torch.bfloat16)
    xq, wq = moeq.moeq_quantize_mxfp4(x), moeq.moeq_quantize_mxfp4(w)
    a = _f64(moeq.moeq_grouped_mm_mxfp4(xq, wq, off))
    xd, wd = moeq.moeq_dequantize(xq)[0], moeq.moeq_dequantize(wq)
    b = _f64(moeq.moeq_grouped_mm(xd, wd, off))
    mag = grouped_mm(np.abs(_f64(xd)), np.abs(_f64(wd)), host(off))
    # the same exact products: two fp32 sums of 288 terms, two roundings
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b) * (1 + 2.0 ** -7) + 2 * 288 * 2.0 ** -23 * mag * (1 + 2.0 ** -7)).all()


def test_operands_past_32_bit_offsets():
    """x, w and the outputs of more than 2^32 bytes: the last rows and the last
    expert against fp64."""
    say("grouped large")
    g = torch.Generator(device=DEV).manual_seed(31)

    def check(got, a, b, L):   # got = a @ b^T
        a, b = a.double(), b.double()
        want, mag = a @ b.t(), a.abs() @ b.abs().t()
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + L * 2.0 ** -23 * mag * (1 + 2.0 ** -8)).all())

    M, N, K, E = (1 << 20) + 77, 16, 2056, 3   # x: 4.3 GB; long experts, narrow output
    x = torch.randn((M, K), generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.randn((E, N, K), generator=g, device=DEV, dtype=torch.bfloat16)
    off = torch.tensor([0, 1000, M - 300, M], dtype=torch.int32, device=DEV)
    check(moeq.moeq_grouped_mm(x, w, off)[-300:], x[-300:], w[2], K)
    dy = torch.randn((M, N), generator=g, device=DEV, dtype=torch.bfloat16)
    check(moeq.moeq_grouped_mm_grad_input(dy, w, off)[-300:], dy[-300:], w[2].t(), N)
    dw = moeq.moeq_grouped_mm_grad_weight(dy, x, off)
    check(dw[2], dy[-300:].t(), x[-300:].t(), 300)
    xq, wq = moeq.moeq_quantize_mxfp4(torch.randn((M, 8192), generator=g, device=DEV, dtype=torch.bfloat16)), \
        moeq.moeq_quantize_mxfp4(torch.randn((E, 24, 8192), generator=g, device=DEV, dtype=torch.bfloat16))
    y = moeq.moeq_grouped_mm_mxfp4(xq, wq, off)      # codes: 4.3 GB
    tail = moeq.QWeight(moeq.FMT_MXFP4, 1, 300, 8192, xq.qdata[:, -300:].contiguous(), None,
                        xq.scale_codes[:, -300:].contiguous())
    check(y[-300:], moeq.moeq_dequantize(tail)[0], moeq.moeq_dequantize(wq)[2], 8192)
    del x, dy, xq, dw
    E, N, K = 35, 8192, 8192                          # w: 4.7 GB
    w = torch.randn((E, N, K), generator=g, device=DEV, dtype=torch.bfloat16)
    for rows in (3, 70):                              # weight streaming, and tiles
        off = torch.arange(E + 1, dtype=torch.int32, device=DEV) * rows
        x = torch.randn((E * rows, K), generator=g, device=DEV, dtype=torch.bfloat16)
        check(moeq.moeq_grouped_mm(x, w, off)[-rows:], x[-rows:], w[-1], K)
        check(moeq.moeq_grouped_mm_grad_input(x, w, off)[-rows:], x[-rows:], w[-1].t(), N)
    dw = moeq.moeq_grouped_mm_grad_weight(x, x, off, dtype=torch.bfloat16)
    check(dw[-1], x[-70:].t(), x[-70:].t(), 70)
