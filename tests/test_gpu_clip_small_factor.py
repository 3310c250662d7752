"""GPU: gradient clipping whose factor max_norm / norm lies below fp32's
smallest normal number (large gradients, a small max_norm).  The bounds are
those of every other factor: 2^-24 for the factor, 2^-24 for the product, and
2^-8 more for bf16; the results themselves are normal numbers."""

import math

import numpy as np
import pytest
import torch

import bit_weight_quantization_moeq_amd as moeq
from tests.gpu_common import DEV, host, require_native, say
from tests.test_gpu_clip import _check, _grads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _native():
    require_native()


@pytest.mark.parametrize("std,max_norm", [(1e36, 1e-3), (1e35, 2.5),   # (2.5: still a normal factor)
                                          (3e35, 1e-7), (1e34, 1e-30), (2.0 ** 100, 2.0 ** -40)])
def test_factor_near_and_below_fp32_normal_numbers(std, max_norm):
    say(f"clip factor {std} {max_norm}")
    grads = _grads([3001, 77, 20000], [torch.float32, torch.bfloat16], seed=5, std=std)
    keep = [g.clone() for g in grads]
    out = [torch.full_like(g, 7.0) for g in grads]
    norm = moeq.moeq_clip_grad_norm(grads, max_norm, out=out)
    assert math.isfinite(float(norm))
    _check(keep, out, norm, max_norm)
    assert torch.equal(moeq.moeq_clip_grad_norm(grads, max_norm), norm)   # in place
    assert all(torch.equal(a, b) for a, b in zip(grads, out))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_past_fp32_reads_as_an_infinity_and_still_clips(dtype):
    """64 equal gradients v have the norm 8 v: below, and past, fp32's range."""
    say(f"clip norm past fp32 {dtype}")
    for v, finite in ((2.0 ** 124, True), (2.0 ** 125, False), (2.0 ** 127, False)):
        g = [torch.full((40,), v, dtype=dtype, device=DEV), torch.full((24,), -v, dtype=dtype, device=DEV)]
        out = [torch.full_like(t, 7.0) for t in g]
        norm = moeq.moeq_clip_grad_norm(g, 2.0 ** 120, out=out)
        assert float(norm) == (8 * v if finite else math.inf)
        assert (out[0] == 2.0 ** 117).all() and (out[1] == -(2.0 ** 117)).all()   # v 2^120 / (8 v)


def test_results_below_fp32_normal_numbers():
    """A factor and results that are subnormal, or too small for either."""
    say("clip tiny results")
    for max_norm in (1e-40, 1e-300):
        grads = _grads([1000, 500], [torch.float32, torch.bfloat16], seed=6, std=1e30)
        keep = [g.clone() for g in grads]
        norm = moeq.moeq_clip_grad_norm(grads, max_norm)
        _check(keep, grads, norm, max_norm)
        for g, k in zip(grads, keep):
            gone = np.abs(host(k.double())) * (max_norm / float(norm)) < 2.0 ** -151
            assert not host(g.double())[gone].any()
