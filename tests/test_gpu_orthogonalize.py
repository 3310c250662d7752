"""GPU: orthogonalised updates against the 64-bit oracle.

The bound is one on the 2-norm of a matrix's whole error, followed step by step
through the exact iterates in 64 bits.  A value kept in fp16 is off by 2^-11 of
itself (or 2^-25 of the power of two it is stored with), an fp32 sum of L products
by L 2^-23 of the sum of their magnitudes.  With |.| the 2-norm of a matrix's
entries and ||.|| its largest singular value, one step adds
  dA = 2^-11 |A| + L 2^-23 | |X||X^T| |
  dP = (|b| + 2 |c| ||A||) dA + 2^-11 |P| + (n + 4) 2^-23 (|a| sqrt(n) + |b| |A| + |c| | |A||A| |)
  dX = dP ||X|| + 2^-11 |X'| + n 2^-23 | |P||X| |
to its result.  An error E of its input reaches the result through the step's
derivative, which in the exact iterate's singular basis multiplies the entries of
E's symmetric part by (f(s) - f(t)) / (s - t), those of its antisymmetric part by
(f(s) + f(t)) / (s + t), and what lies outside the shorter side's space by f(s) / s,
with s, t the singular values and f(s) = a s + b s^3 + c s^5: at most the largest of
these.  The output's rounding to bf16 is 2^-8 of it.  Second-order terms are below
a tenth of this: 1.1.

That is the worst case, 6 to 40 % of the result.  Matrices of 64 entries and more
are held to what to expect, too: roundings are independent and spread evenly over
the half steps (the 2-norm over the square root of 3), an error matrix has no
direction of its own, so that squares add, a step multiplies by the factors' root
mean square over all entries, and |E X| is |E| |X| / sqrt(n) for a random n x n E.
Three times that (sums over 64 entries and more stray far less).  It grows with
missing directions, whose rounding a step multiplies by a as it does small singular
values: a matrix of rank one is 10 % off after five steps, one of full rank 0.2 %."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from oracle.orthogonalize import COEFFICIENTS, orthogonalize, start, step
from tests.gpu_common import DEV, require_native, say
from tests.test_gpu_grouped import _f64
from tests.test_gpu_guarded import Guarded

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
H, S = 2.0 ** -11, 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _norm(m):
    return float(np.sqrt((np.asarray(m) ** 2).sum()))


def _factors(s, abc, m):
    """Of the factors by which a step multiplies the parts of its input's error:
    the largest, and the root mean square over n x m entries."""
    a, b, c = abc
    s, t = s[:, None], s[None, :]
    # (f(s) -+ f(t)) / (s -+ t) without the quotient
    minus = a + b * (s * s + s * t + t * t) + c * (s ** 4 + s ** 3 * t + s * s * t * t + s * t ** 3 + t ** 4)
    plus = a + b * (s * s - s * t + t * t) + c * (s ** 4 - s ** 3 * t + s * s * t * t - s * t ** 3 + t ** 4)
    out = a + b * s * s + c * s ** 4
    n = minus.shape[0]
    mean = (((minus ** 2 + plus ** 2) / 2).sum() + (m - n) * (out ** 2).sum()) / (n * m)
    return max(np.abs(minus).max(), np.abs(plus).max(), np.abs(out).max()), np.sqrt(mean)


def _bound(g, table):
    """What the result may be off by at most, what to expect, and the exact result."""
    x = start(g)
    if x.shape[0] > x.shape[1]:
        x = x.T
    n, m = x.shape
    tiny = 2.0 ** -25 * 2.0 ** -min(15, int(np.log2(m) / 2))
    err = H * _norm(x) + tiny * np.sqrt(n * m)
    rms, even = err / np.sqrt(3), H / np.sqrt(3)
    for a, b, c in table:
        A = x @ x.T
        A2, P = A @ A, a * np.eye(n) + b * A
        P = P + c * A2
        y = step(x, (a, b, c))
        values = np.linalg.svd(x, compute_uv=False)
        top, topA = values[0], values[0] ** 2
        dA = H * _norm(A) + m * S * _norm(np.abs(x) @ np.abs(x.T)) + 2.0 ** -33 * n
        dP = (abs(b) + 2 * abs(c) * topA) * dA + H * _norm(P) + 2.0 ** -33 * n
        dP += (n + 4) * S * (abs(a) * np.sqrt(n) + abs(b) * _norm(A) + abs(c) * _norm(np.abs(A) @ np.abs(A)))
        dX = dP * top + H * _norm(y) + n * S * _norm(np.abs(P) @ np.abs(x)) + tiny * np.sqrt(n * m)
        most, mean = _factors(values, (a, b, c), m)
        err = err * most + dX
        lam = values ** 2
        poly = np.sqrt(np.mean((b + c * (lam[:, None] + lam[None, :])) ** 2)) * even * _norm(A)
        rms = np.sqrt((rms * mean) ** 2 + (poly ** 2 + (even * _norm(P)) ** 2) * _norm(x) ** 2 / n + (even * _norm(y)) ** 2)
        x = y
    expected = np.sqrt(rms ** 2 + (2.0 ** -8 * _norm(x)) ** 2 / 3)
    return 1.1 * err + 2.0 ** -8 * _norm(x), expected, x if np.shape(g)[0] <= np.shape(g)[1] else x.T


def _check(g, out, table=(COEFFICIENTS,) * 5):
    g, out = _f64(g), _f64(out)
    for e in range(g.shape[0]):
        tol, expected, want = _bound(g[e], table)
        off = _norm(out[e] - want)
        assert off <= tol, (e, off, tol)
        assert want.size < 64 or off <= 3 * expected, (e, off, expected, _norm(want))


SHAPES = [(1, 1, 1), (2, 1, 300), (2, 300, 1), (3, 3, 3), (3, 16, 72), (2, 72, 16), (2, 40, 41), (2, 41, 40), (2, 64, 64),
          (1, 65, 1000), (1, 1000, 65), (2, 129, 257), (1, 257, 129), (1, 264, 264), (1, 300, 515), (5, 16, 2048), (1, 520, 300)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_the_oracle(shape, dtype):
    say(f"orthogonalize {shape} {dtype}")
    g = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(dtype)
    out = moeq.moeq_orthogonalize(g)
    assert out.dtype == BF16 and out.shape == g.shape
    _check(g, out)
    assert torch.equal(out, moeq.moeq_orthogonalize(g))
    if shape[0] == 1:
        assert torch.equal(out[0], moeq.moeq_orthogonalize(g[0]))


def test_each_tile_shape():
    """Enough matrices for the tiles of 64, 128 and 256 to be the ones that run."""
    for shape in ((40, 200, 328), (40, 328, 200), (70, 300, 520), (70, 520, 300)):
        say(f"orthogonalize tiles {shape}")
        g = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(BF16)
        out = moeq.moeq_orthogonalize(g)
        pick = [0, 17, shape[0] - 1]
        _check(g[pick], out[pick])
        for e in (0, shape[0] - 1):   # alone, in other tiles: the same sums in the same order
            one = moeq.moeq_orthogonalize(g[e])
            assert (one.float() - out[e].float()).norm() <= 2.0 ** -6 * out[e].float().norm()


@pytest.mark.parametrize("factor", [1e-38, 1e-20, 1.0, 1e18, 1e30])
def test_the_length_does_not_matter(factor):
    say(f"orthogonalize length {factor}")
    g = torch.randn((2, 48, 80), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    _check(g * factor, moeq.moeq_orthogonalize(g * factor))


def test_known_singular_values():
    say("orthogonalize singular values")
    r = np.random.default_rng(4)
    u, _ = np.linalg.qr(r.standard_normal((96, 96)))
    v, _ = np.linalg.qr(r.standard_normal((160, 160)))
    s = np.geomspace(1.0, 0.02, 96)
    g = torch.from_numpy((u * s) @ v[:96]).float().to(DEV)[None]
    out = moeq.moeq_orthogonalize(g)
    _check(g, out)
    got = np.linalg.svd(_f64(out)[0], compute_uv=False)
    assert 0.6 < got.min() and got.max() < 1.3


@pytest.mark.parametrize("steps,table", [(1, (1.5, -0.5, 0.0)), (3, [(4.0, -6.0, 2.5), (3.0, -4.0, 2.0), (1.5, -0.5, 0.0)]),
                                         (6, (1.875, -1.25, 0.375))])
def test_other_coefficients(steps, table):
    say(f"orthogonalize coefficients {table}")
    g = torch.randn((2, 72, 200), generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(BF16)
    rows = table if isinstance(table, list) else [table] * steps
    _check(g, moeq.moeq_orthogonalize(g, steps, table), rows)


def test_zeros_infinities_and_nans_stay_in_their_matrix():
    say("orthogonalize bad matrices")
    for shape in ((6, 40, 72), (6, 72, 40), (6, 16, 264)):
        g = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)
        ref = moeq.moeq_orthogonalize(g)
        g[1] = 0
        g[2, 3, 5], g[4, -1, -1] = float("inf"), float("nan")
        out = moeq.moeq_orthogonalize(g)
        assert not out[1].any() and out[2].isnan().all() and out[4].isnan().all()
        for e in (0, 3, 5):
            assert torch.equal(out[e], ref[e])


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 5, 7), (2, 16, 264), (2, 130, 72), (3, 33, 100), (1, 264, 520), (2, 300, 515)])
def test_nothing_is_written_past_the_end(shape):
    say(f"orthogonalize guarded {shape}")
    g = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(7), device=DEV)
    out, ws = Guarded(shape, BF16), Guarded((moeq.moeq_orthogonalize_workspace_bytes(*shape),), U8, 0xff)
    assert torch.equal(moeq.moeq_orthogonalize(g, out=out.t, workspace=ws.t), moeq.moeq_orthogonalize(g))
    out.check("out")
    ws.check("workspace")


def test_an_input_at_any_float():
    say("orthogonalize unaligned")
    flat = torch.randn(2 * 24 * 40 + 3, generator=torch.Generator(device=DEV).manual_seed(8), device=DEV)
    for dtype in (F32, BF16):
        f = flat.to(dtype)
        g = f[3:].view(2, 24, 40)
        assert torch.equal(moeq.moeq_orthogonalize(g), moeq.moeq_orthogonalize(g.clone()))


def test_empty():
    say("orthogonalize empty")
    for shape in ((0, 4, 4), (2, 0, 4), (2, 4, 0), (0, 8)):
        assert moeq.moeq_orthogonalize(torch.empty(shape, device=DEV)).shape == shape


def test_other_stream_and_graph():
    say("orthogonalize stream, graph")
    g = torch.randn((3, 72, 136), generator=torch.Generator(device=DEV).manual_seed(9), device=DEV)
    ref = moeq.moeq_orthogonalize(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moeq.moeq_orthogonalize(g, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moeq.moeq_orthogonalize(g)
    for k in range(4):
        g.copy_(torch.randn(g.shape, generator=torch.Generator(device=DEV).manual_seed(k), device=DEV))
        ref = moeq.moeq_orthogonalize(g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, ref), k


def test_oracle_side():
    """(the bound's exact result is the oracle's)"""
    g = np.random.default_rng(10).standard_normal((12, 7))
    assert np.allclose(_bound(g, (COEFFICIENTS,) * 5)[2], orthogonalize(g), atol=1e-12)


# (rows up to 16 and up to 32, either side long, columns up to 2048 and beyond, and what is past them)
@pytest.mark.parametrize("shape", [(2, 16, 2049), (2, 2500, 9), (1, 16, 8192), (1, 8192, 16), (1, 13, 8193), (3, 17, 2048),
                                   (2, 32, 2049), (1, 4096, 32), (1, 4097, 31), (300, 7, 130), (2, 33, 2048)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_rows(shape, dtype):
    say(f"orthogonalize few rows {shape} {dtype}")
    g = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(11), device=DEV).to(dtype)
    out = Guarded(shape, BF16)
    moeq.moeq_orthogonalize(g, out=out.t)
    out.check("out")
    pick = [0, shape[0] - 1]
    _check(g[pick], out.t[pick])
    assert torch.equal(out.t, moeq.moeq_orthogonalize(g))


@pytest.mark.parametrize("shape", [(3, 64, 16), (3, 16, 64), (2, 72, 12), (2, 2048, 16), (1, 4096, 32), (2, 9, 200), (2, 130, 300),
                                   (2, 300, 130)])
@pytest.mark.parametrize("rank", [1, 3, 1000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ranks(shape, rank, dtype):
    """Gradients of experts with few rows have few directions."""
    say(f"orthogonalize {shape} rank {rank} {dtype}")
    gen = torch.Generator(device=DEV).manual_seed(12)
    E, N, K = shape
    r = min(rank, N, K)
    u, v = (torch.randn(s, generator=gen, device=DEV) for s in ((E, N, r), (E, r, K)))
    g = (torch.randn(shape, generator=gen, device=DEV) if rank == 1000 else u @ v).to(dtype)
    _check(g, moeq.moeq_orthogonalize(g))


def test_one_entry_at_a_time():
    """With (a, b, c) = (1, 0, 0) the update is G / |G|: every entry keeps its place."""
    say("orthogonalize places")
    for N, K in ((20, 4), (4, 20), (64, 16), (32, 40), (40, 32), (70, 90)):
        for dtype in (BF16, F32):
            g = torch.zeros((N * K, N, K), dtype=dtype, device=DEV)
            g.view(N * K, N * K).fill_diagonal_(3.0)
            g = g[::7].contiguous()
            assert torch.equal(moeq.moeq_orthogonalize(g, 1, (1.0, 0.0, 0.0)), (g / 3).to(BF16)), (N, K, dtype)
