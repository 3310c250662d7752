"""GPU: the experts' gated feed-forward block and its gradients against the
64-bit oracle, output by output.

Tolerances, from the arithmetic.  An fp32 sum of L exact products is off by at
most L 2^-23 of the sum of their magnitudes (the matrix cores may truncate).
exp and the reciprocal are off by some units of 2^-23, exp's argument by |g|
more; every formula below has at most ten operations, so kOps = 16 of them are
allowed.  A value stored in bf16 is off by 2^-8 of itself.  With s the sigmoid:
  g, u     |d| <= H 2^-23 mag (saved as they are)
  h        |u s (1 + g (1 - s))| dg + |g s| du + (kOps + |g|) 2^-23 |h|, then 2^-8
  dg, du   the same with dh's error (H 2^-23 mag) and the sum's two terms apart
  out, grad_x and the weights' gradients: the products of the operands' errors
           and the others' magnitudes, an fp32 sum, then a rounding to the type.
The backward pass is compared with the oracle on the g and u that were saved,
which are its input."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from oracle.ffn import activation_gradients, ffn_backward, hidden, pre_activations, sigmoid
from oracle.grouped import grouped_mm, grouped_mm_grad_input, grouped_mm_grad_weight
from tests.gpu_common import DEV, require_native, say
from tests.test_gpu_grouped import ROWS, _clean, _f64, _offsets, _untouched
from tests.test_gpu_guarded import Guarded

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
SUM, HALF, OPS = 2.0 ** -23, 2.0 ** -8, 16
SHAPES = [(8, 8), (64, 16), (72, 136), (264, 520), (520, 264), (1032, 40), (136, 1000)]


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _case(sizes, before, behind, H, I, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    off = _offsets(sizes, before)
    M, E = int(off[-1]) + behind, len(sizes)
    x, dy = (torch.randn((M, H), generator=g, device=DEV).to(BF16) for _ in range(2))
    w1 = (torch.randn((E, 2 * I, H), generator=g, device=DEV) * 1.5 * H ** -0.5).to(BF16)
    w2 = (torch.randn((E, H, I), generator=g, device=DEV) * I ** -0.5).to(BF16)
    for t in (x, dy):   # rows of no expert hold anything
        t[:off[0]] = float("nan")
        t[off[-1]:] = float("inf")
    return x, dy, w1, w2, off, torch.from_numpy(off).to(DEV)


def _near(got, want, tol, label):
    got = _f64(got)
    live = ~np.isnan(want)
    bad = live & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (label, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


def _check_forward(x, w1, w2, off, y, gu):
    H, I = w2.shape[1], w2.shape[2]
    xs, a, b = _clean(x, off), _f64(w1), _f64(w2)
    want = pre_activations(xs, a, off)
    err = H * SUM * pre_activations(np.abs(xs), np.abs(a), off)
    if gu is not None:
        _near(gu, want, err, "gu")
    g, u = np.split(want, 2, axis=1)
    eg, eu = np.split(err, 2, axis=1)
    s, h = sigmoid(g), hidden(want)
    # (the derivative where g is off by eg: within a factor of 1 + eg)
    eh = (np.abs(u) * s * (1 + np.abs(g) * (1 - s)) * eg + np.abs(g) * s * eu + eg * eu) * (1 + eg)
    eh = eh + (OPS + np.abs(g)) * SUM * np.abs(h)
    eh = eh + HALF * (np.abs(h) + eh)
    out = grouped_mm(h, b, off)
    tol = grouped_mm(eh, np.abs(b), off) + I * SUM * grouped_mm(np.abs(h) + eh, np.abs(b), off)
    _near(y, out, HALF * np.abs(out) + tol * (1 + HALF), "out")


def _check_backward(dy, x, w1, w2, off, gu, grads, half):
    H, I = w2.shape[1], w2.shape[2]
    xs, d, a, b, p = _clean(x, off), _clean(dy, off), _f64(w1), _f64(w2), _clean(gu, off)
    want = ffn_backward(d, xs, a, b, off, p)
    g, u = np.split(p, 2, axis=1)
    s = sigmoid(g)
    dh = grouped_mm_grad_input(d, b, off)
    ed = H * SUM * grouped_mm_grad_input(np.abs(d), np.abs(b), off)
    both = np.concatenate([np.abs(u) * s * (1 + np.abs(g) * (1 - s)), np.abs(g) * s], axis=1)
    dgu = activation_gradients(dh, p)
    e = np.concatenate([ed, ed], 1) * both + np.concatenate([(np.abs(dh) + ed) * (OPS + np.abs(g))] * 2, 1) * SUM * both
    e = e + HALF * (np.abs(dgu) + e)
    h = hidden(p)
    eh = (HALF + (OPS + np.abs(g)) * SUM) * np.abs(h)
    dx, dw1, dw2 = grads
    tol = grouped_mm_grad_input(e, np.abs(a), off)
    tol = tol + 2 * I * SUM * grouped_mm_grad_input(np.abs(dgu) + e, np.abs(a), off)
    _near(dx, want[0], HALF * np.abs(want[0]) + tol * (1 + HALF), "grad_x")
    L = int(np.diff(off).max())
    z = lambda t: np.nan_to_num(t)   # (rows of no expert)  # noqa: E731
    tol = grouped_mm_grad_weight(z(e), np.abs(xs), off) + L * SUM * grouped_mm_grad_weight(z(np.abs(dgu) + e), np.abs(xs), off)
    _near(dw1, want[1], half * np.abs(want[1]) + tol * (1 + half), "grad_gate_up")
    tol = grouped_mm_grad_weight(np.abs(d), z(eh), off) + L * SUM * grouped_mm_grad_weight(np.abs(d), z(np.abs(h) + eh), off)
    _near(dw2, want[2], half * np.abs(want[2]) + tol * (1 + half), "grad_down")


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("H,I", SHAPES)
def test_block_and_gradients(rows, H, I):
    say(f"ffn {rows} H={H} I={I}")
    x, dy, w1, w2, off, doff = _case(*ROWS[rows], H, I)
    M = x.shape[0]
    y, gu = torch.full((M, H), 7.0, dtype=BF16, device=DEV), torch.full((M, 2 * I), 7.0, dtype=F32, device=DEV)
    got = moeq.moeq_grouped_ffn(x, w1, w2, doff, out=y, gu=gu)
    assert got[0] is y and got[1] is gu
    _check_forward(x, w1, w2, off, y, gu)
    assert _untouched(y, off) and _untouched(gu, off)
    plain = moeq.moeq_grouped_ffn(x, w1, w2, doff)      # without saving: the same bits
    assert torch.equal(plain[off[0]:off[-1]], y[off[0]:off[-1]])

    gu[:off[0]], gu[off[-1]:] = float("nan"), float("inf")
    for dtype, half in ((F32, 2.0 ** -24), (BF16, HALF)):
        dx = torch.full((M, H), 7.0, dtype=BF16, device=DEV)
        grads = moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, doff, gu, dtype=dtype, grad_x=dx)
        assert grads[0] is dx and grads[1].dtype == grads[2].dtype == dtype
        _check_backward(dy, x, w1, w2, off, gu, grads, half)
        assert _untouched(dx, off)
        for e in np.flatnonzero(np.diff(off) == 0):
            assert not grads[1][e].any() and not grads[2][e].any()


@pytest.mark.parametrize("sizes", [[1500], [0, 513, 1, 512, 2050, 0, 700]])
def test_long_experts(sizes):
    say(f"ffn long {sizes}")
    x, dy, w1, w2, off, doff = _case(sizes, 3, 2, 264, 136, seed=5)
    y, gu = moeq.moeq_grouped_ffn(x, w1, w2, doff, save=True)
    _check_forward(x, w1, w2, off, y, gu)
    grads = moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, doff, gu)
    _check_backward(dy, x, w1, w2, off, gu, grads, 2.0 ** -24)
    for a, b in zip(grads, moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, doff, gu)):
        assert torch.equal(a[off[0]:off[-1]] if a is grads[0] else a, b[off[0]:off[-1]] if a is grads[0] else b)


def test_far_gates():
    """Gates far outside exp's range: silu is 0 or the gate itself."""
    say("ffn far gates")
    H = I = 8
    x = torch.eye(8, device=DEV).to(BF16) * 100
    w1 = torch.zeros((1, 16, 8), device=DEV)
    w1[0, 0, :] = torch.tensor([-100.0, -1.0, -0.5, 0.0, 0.5, 1.0, 100.0, 2.0 ** 60])
    w1[0, 8, :] = 1.0
    w2 = torch.zeros((1, 8, 8), device=DEV)
    w2[0, 0, 0] = 1.0
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    y, gu = moeq.moeq_grouped_ffn(x, w1.to(BF16), w2.to(BF16), off, save=True)
    want = hidden(_f64(gu))[:, 0]
    # the roundings of h and of the output
    assert np.all(np.abs(_f64(y)[:, 0] - want) <= 2.1 * HALF * np.abs(want) + 1e-30)
    dx, dw1, dw2 = moeq.moeq_grouped_ffn_backward(torch.ones_like(x), x, w1.to(BF16), w2.to(BF16), off, gu)
    assert all(torch.isfinite(t).all() for t in (dx, dw1, dw2))


def test_no_rows():
    say("ffn no rows at all")
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    x, gu = torch.empty((0, 16), dtype=BF16, device=DEV), torch.empty((0, 48), dtype=F32, device=DEV)
    w1, w2 = torch.ones((2, 48, 16), dtype=BF16, device=DEV), torch.ones((2, 16, 24), dtype=BF16, device=DEV)
    assert moeq.moeq_grouped_ffn(x, w1, w2, off).shape == (0, 16)
    dx, dw1, dw2 = moeq.moeq_grouped_ffn_backward(x, x, w1, w2, off, gu)
    assert dx.shape == (0, 16) and not dw1.any() and not dw2.any()


GUARDED = {"one row": [1], "few": [2, 0, 9, 1, 17, 0, 3, 8], "borders": [32, 64, 65, 128, 129, 192, 193, 256, 257],
           "long": [40] * 20 + [1500], "many experts": [(i * 7) % 40 + 1 for i in range(300)]}


@pytest.mark.parametrize("rows", list(GUARDED))
@pytest.mark.parametrize("H,I", [(8, 8), (264, 16), (72, 136), (1032, 200)])
def test_nothing_is_written_past_the_end(rows, H, I):
    say(f"ffn guarded {rows} H={H} I={I}")
    x, dy, w1, w2, off, doff = _case(GUARDED[rows], 0, 0, H, I, seed=2)
    M, E = x.shape[0], len(off) - 1
    y, gu = Guarded((M, H), BF16), Guarded((M, 2 * I), F32)
    ws = Guarded((moeq.moeq_grouped_ffn_workspace_bytes(M, E, H, I),), U8)
    moeq.moeq_grouped_ffn(x, w1, w2, doff, out=y.t, gu=gu.t, workspace=ws.t)
    ref = moeq.moeq_grouped_ffn(x, w1, w2, doff, save=True)
    assert torch.equal(y.t, ref[0]) and torch.equal(gu.t, ref[1])
    for t in (y, gu, ws):
        t.check("forward")
    dx, bw = Guarded((M, H), BF16), Guarded((moeq.moeq_grouped_ffn_backward_workspace_bytes(M, E, H, I),), U8)
    for dtype in (F32, BF16):
        dw1, dw2 = Guarded((E, 2 * I, H), dtype), Guarded((E, H, I), dtype)
        moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, doff, gu.t, grad_x=dx.t, grad_gate_up=dw1.t, grad_down=dw2.t,
                                       workspace=bw.t)
        want = moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, doff, gu.t, dtype=dtype)
        for t, v in zip((dx, dw1, dw2), want):
            assert torch.equal(t.t, v)
            t.check("backward")
        bw.check("workspace")


@pytest.mark.parametrize("bad", [[0, 40, 20, 50], [-2 ** 31, 70, -5, 2 ** 31 - 1], [60, 0, 60, 0], [2 ** 31 - 1] * 4])
def test_offsets_that_do_not_ascend_stay_inside(bad):
    say(f"ffn offsets {bad}")
    x, dy, w1, w2, _, _ = _case([20, 20, 20], 0, 0, 72, 40, seed=3)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    y, gu = Guarded((60, 72), BF16, 1.0), Guarded((60, 80), F32, 1.0)
    ws, bw = (Guarded((n(60, 3, 72, 40),), U8) for n in (moeq.moeq_grouped_ffn_workspace_bytes,
                                                         moeq.moeq_grouped_ffn_backward_workspace_bytes))
    moeq.moeq_grouped_ffn(x, w1, w2, off, out=y.t, gu=gu.t, workspace=ws.t)
    dx, dw1, dw2 = Guarded((60, 72), BF16), Guarded((3, 80, 72), F32), Guarded((3, 72, 40), F32)
    moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, off, gu.t, grad_x=dx.t, grad_gate_up=dw1.t, grad_down=dw2.t,
                                   workspace=bw.t)
    for t in (y, gu, ws, bw, dx, dw1, dw2):
        t.check("offsets")


def test_other_stream_and_graph():
    """On a stream of its own, and captured: every replay on new inputs equals the eager call."""
    say("ffn stream, graph")
    x, dy, w1, w2, off, doff = _case([5, 0, 130, 33], 0, 0, 136, 72, seed=4)

    def step():
        y, gu = moeq.moeq_grouped_ffn(x, w1, w2, doff, save=True)
        return (y, *moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, doff, gu, dtype=BF16))

    ref = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, gu = moeq.moeq_grouped_ffn(x, w1, w2, doff, save=True, stream=s)
    got = (y, *moeq.moeq_grouped_ffn_backward(dy, x, w1, w2, doff, gu, dtype=BF16, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device=DEV).manual_seed(k), device=DEV))
        ref = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), k
