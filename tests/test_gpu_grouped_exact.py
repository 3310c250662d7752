"""GPU: grouped products on operands whose products and sums are exact, so
that every result has to be the exact one, rounded once: a single contraction
element that is lost, doubled or taken from a neighbour shows.

bf16: integers of magnitude 8 at most, so sums of up to 2^18 products are
integers below 2^24, exact in fp32 in any order.  MXFP4: E2M1 values (multiples
of 1/2, 6 at most) under scales 1 and 2, so products are multiples of 1/4 of
magnitude 144 at most, and sums of up to 2^14 of them are exact, too.

The shapes reach every form of the tiles: those of 256 x 256 (wider outputs
than 128 tiles' worth) with one to four blocks of 32 rows a wave, those of a
contraction of one step, column and contraction tails, one step to many, and
more experts than one pass of the expert search takes (256)."""

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from oracle.mxfp4 import mxfp4_dequantize
from tests.gpu_common import DEV, host, require_native, say

pytestmark = pytest.mark.gpu

BEFORE, BEHIND = 3, 5   # rows of no expert


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


def _offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + np.int32(BEFORE)


def _ints(shape, g):
    return torch.randint(-8, 9, shape, generator=g, device=DEV).to(torch.bfloat16)


def _rows(M, cols, off, g):
    t = _ints((M, cols), g)
    t[:BEFORE], t[off[-1]:] = float("nan"), float("inf")
    return t


def _same_rows(got, off, want_of):
    """got's rows of expert e are want_of(e, lo, hi) rounded to bf16, the rest 7."""
    want = torch.full_like(got, 7.0)
    for e in range(len(off) - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            want[lo:hi] = want_of(e, lo, hi).to(torch.bfloat16)
    bad = (got != want).nonzero()
    assert bad.shape[0] == 0, (bad.shape[0], bad[:4].tolist(), [(float(got[tuple(i)]), float(want[tuple(i)])) for i in bad[:4]])


def _forward(sizes, nout, kc, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    off = _offsets(sizes)
    M = int(off[-1]) + BEHIND
    x, w = _rows(M, kc, off, g), _ints((len(sizes), nout, kc), g)
    y = torch.full((M, nout), 7.0, dtype=torch.bfloat16, device=DEV)
    moeq.moeq_grouped_mm(x, w, torch.from_numpy(off).to(DEV), out=y)
    _same_rows(y, off, lambda e, lo, hi: x[lo:hi].double() @ w[e].double().t())


def _grad_input(sizes, nout, kc, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    off = _offsets(sizes)
    M = int(off[-1]) + BEHIND
    dy, w = _rows(M, kc, off, g), _ints((len(sizes), kc, nout), g)
    dx = torch.full((M, nout), 7.0, dtype=torch.bfloat16, device=DEV)
    moeq.moeq_grouped_mm_grad_input(dy, w, torch.from_numpy(off).to(DEV), grad_x=dx)
    _same_rows(dx, off, lambda e, lo, hi: dy[lo:hi].double() @ w[e].double())


def _grad_weight(sizes, N, K, seed=2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    off = _offsets(sizes)
    M = int(off[-1]) + BEHIND
    dy, x = _rows(M, N, off, g), _rows(M, K, off, g)
    doff = torch.from_numpy(off).to(DEV)
    dw = moeq.moeq_grouped_mm_grad_weight(dy, x, doff)
    for e in range(len(sizes)):
        lo, hi = int(off[e]), int(off[e + 1])
        assert torch.equal(dw[e].double(), dy[lo:hi].double().t() @ x[lo:hi].double()), (e, sizes[e])
    assert torch.equal(moeq.moeq_grouped_mm_grad_weight(dy, x, doff, dtype=torch.bfloat16), dw.to(torch.bfloat16))


def _mx(shape, g):
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(127, 129, (*shape[:-1], shape[-1] // 32), generator=g, device=DEV, dtype=torch.uint8)
    values = torch.from_numpy(mxfp4_dequantize(host(codes), host(scales))).to(DEV)
    return moeq.QWeight(moeq.FMT_MXFP4, *shape, codes, None, scales), values


def _mxfp4(sizes, nout, kc, seed=3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    off = _offsets(sizes)
    M = int(off[-1]) + BEHIND
    (xq, x), (wq, w) = _mx((1, M, kc), g), _mx((len(sizes), nout, kc), g)
    xq.scale_codes[0, :BEFORE], xq.scale_codes[0, off[-1]:] = 255, 255   # NaN
    y = torch.full((M, nout), 7.0, dtype=torch.bfloat16, device=DEV)
    moeq.moeq_grouped_mm_mxfp4(xq, wq, torch.from_numpy(off).to(DEV), out=y)
    _same_rows(y, off, lambda e, lo, hi: x[0, lo:hi] @ w[e].t())


# Rows of a 256-row tile around every number of 32-row blocks, and more than one tile.
TILE_ROWS = [250, 190, 120, 60, 257, 0, 256, 1, 129, 193, 64, 65, 128, 192, 33, 600]
SIZES = [TILE_ROWS[i % len(TILE_ROWS)] for i in range(40)]


def _tiles_of_256(sizes, nout):
    """As the library estimates them when it chooses the tile (from the number
    of rows and experts); the 256 x 256 tile takes more than 128."""
    M, E = sum(sizes) + BEFORE + BEHIND, len(sizes)
    experts = min(E, M)
    return max(1, (M // experts + 255) // 256) * experts * ((nout + 255) // 256)


WIDE = [2056, 1800]   # nine and eight column tiles, both with tails: 320 and 360 tiles at least


@pytest.mark.parametrize("nout", WIDE)
@pytest.mark.parametrize("kc", [72, 128, 136, 192, 264, 1000])
def test_large_tiles_forward(nout, kc):
    say(f"grouped exact forward {nout} {kc}")
    assert _tiles_of_256(SIZES, nout) >= 2 * 128
    _forward(SIZES, nout, kc)


@pytest.mark.parametrize("nout", WIDE)
@pytest.mark.parametrize("kc", [72, 128, 136, 192, 264, 1000])
def test_large_tiles_grad_input(nout, kc):
    say(f"grouped exact grad_input {nout} {kc}")
    _grad_input(SIZES, nout, kc)


@pytest.mark.parametrize("nout", WIDE)
@pytest.mark.parametrize("kc", [32, 96, 256, 288, 512, 544, 800, 1056])
def test_large_tiles_mxfp4(nout, kc):
    say(f"grouped exact mxfp4 {nout} {kc}")
    _mxfp4(SIZES, nout, kc)


@pytest.mark.parametrize("nout,kc", [(520, 136), (128, 1000), (136, 72), (24, 264)])
def test_narrow_outputs(nout, kc):
    """The tile of 128 columns, for outputs and numbers of experts that leave
    larger ones few, with more than one step."""
    say(f"grouped exact narrow {nout} {kc}")
    sizes = TILE_ROWS
    assert _tiles_of_256(sizes, nout) <= 128
    _forward(sizes, nout, kc)
    _grad_input(sizes, nout, kc)
    _mxfp4(sizes, nout, -(-kc // 32) * 32)


@pytest.mark.parametrize("nout", [8, 72, 264, 2056])
@pytest.mark.parametrize("kc", [8, 16, 24, 40, 56, 64])
def test_contractions_of_one_step(nout, kc):
    say(f"grouped exact short {nout} {kc}")
    _forward(TILE_ROWS, nout, kc)
    _grad_input(TILE_ROWS, nout, kc)


@pytest.mark.parametrize("N,K", [(264, 264), (520, 136), (256, 512), (64, 520), (8, 136), (520, 64), (136, 8), (72, 72), (128, 2056)])
@pytest.mark.parametrize("sizes", [TILE_ROWS, [0, 513, 1, 512, 2050, 0, 700], [3000]])
def test_grad_weight(N, K, sizes):
    say(f"grouped exact grad_weight {N} {K} {len(sizes)}")
    _grad_weight(sizes, N, K)


# Beyond 256 experts the search loads offsets again.
EXPERTS = {
    "300, few rows": [(i * 7) % 5 for i in range(300)],
    "300, tiles": [(i * 7) % 40 for i in range(300)],
    "the first 256 without rows": [0] * 256 + [5, 0, 70, 1, 0, 300],
    "the last one alone": [0] * 511 + [130],
    "1024": [(i * 5) % 23 for i in range(1024)],
    "long ones late": [1] * 260 + [1300, 0, 600, 2],
}


@pytest.mark.parametrize("name", list(EXPERTS))
@pytest.mark.parametrize("nout,kc", [(24, 72), (8, 264), (264, 32), (136, 160)])
def test_more_than_256_experts(name, nout, kc):
    say(f"grouped exact experts {name} {nout} {kc}")
    sizes = EXPERTS[name]
    _forward(sizes, nout, kc)
    _grad_input(sizes, nout, kc)
    _grad_weight(sizes, nout, kc)
    _mxfp4(sizes, nout, -(-kc // 32) * 32)


def _tail(got, want):
    assert torch.equal(got, want.to(got.dtype))


def test_rows_past_32_bit_offsets():
    """x, the outputs and MXFP4 codes of more than 2^32 bytes, in large tiles:
    the last rows."""
    say("grouped exact large rows")
    g = torch.Generator(device=DEV).manual_seed(11)
    M, E = (1 << 20) + 77, 3
    off = torch.tensor([0, 1000, M - 300, M], dtype=torch.int32, device=DEV)
    for nout, kc in ((264, 2056), (2056, 72)):
        x, w = _ints8((M, kc), g), _ints8((E, nout, kc), g)
        _tail(moeq.moeq_grouped_mm(x, w, off)[-700:], torch.cat([x[-700:-300].double() @ w[1].double().t(),
                                                                x[-300:].double() @ w[2].double().t()]))
        wt = w.transpose(1, 2).contiguous()
        _tail(moeq.moeq_grouped_mm_grad_input(x, wt, off)[-300:], x[-300:].double() @ w[2].double().t())
        del x
    codes = torch.randint(0, 256, (1, M, 4096), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(127, 129, (1, M, 256), generator=g, device=DEV, dtype=torch.uint8)
    x = moeq.QWeight(moeq.FMT_MXFP4, 1, M, 8192, codes, None, scales)
    wq, w = _mx((E, 264, 8192), g)
    y = moeq.moeq_grouped_mm_mxfp4(x, wq, off)
    values = torch.from_numpy(mxfp4_dequantize(host(codes[0, -300:]), host(scales[0, -300:]))).to(DEV)
    _tail(y[-300:], values @ w[2].t())


def _ints8(shape, g):
    """As _ints, with less memory on the way."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for s in t.split(max(1, (1 << 28) // t[0].numel())):
        s.copy_(torch.randint(-8, 9, s.shape, generator=g, device=DEV, dtype=torch.int8))
    return t


@pytest.mark.parametrize("rows", [3, 70, 130, 200, 250])
def test_weights_past_32_bit_offsets(rows):
    """w and its gradient of more than 2^32 bytes and long contractions, in the
    streaming form and tiles of one to four blocks a wave: the last expert."""
    say(f"grouped exact large weights {rows}")
    g = torch.Generator(device=DEV).manual_seed(12)
    E, N, K = 35, 8192, 8192
    w = _ints8((E, N, K), g)
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV) * rows
    x = _ints8((E * rows, K), g)
    _tail(moeq.moeq_grouped_mm(x, w, off)[-rows:], x[-rows:].double() @ w[-1].double().t())
    _tail(moeq.moeq_grouped_mm_grad_input(x, w, off)[-rows:], x[-rows:].double() @ w[-1].double())
    dw = moeq.moeq_grouped_mm_grad_weight(x, x, off, grad_w=w)
    _tail(dw[-1], x[-rows:].double().t() @ x[-rows:].double())
