"""The grouped-product oracle against a scalar sum, and its gradients against
central differences of its own forward."""

import numpy as np

from oracle.grouped import grouped_mm, grouped_mm_grad_input, grouped_mm_grad_weight

E, M, N, K = 4, 11, 3, 5
OFF = np.array([1, 4, 4, 9, 10])   # a row before, an expert without rows, a row behind


def _case():
    rng = np.random.default_rng(8)
    return rng.standard_normal((M, K)), rng.standard_normal((E, N, K)), rng.standard_normal((M, N))


def test_forward_against_a_scalar_sum():
    x, w, _ = _case()
    y = grouped_mm(x, w, OFF)
    for p in range(M):
        e = [i for i in range(E) if OFF[i] <= p < OFF[i + 1]]
        for n in range(N):
            if e:
                assert abs(y[p, n] - sum(x[p, k] * w[e[0], n, k] for k in range(K))) < 1e-12
            else:
                assert np.isnan(y[p, n])


def test_gradients_against_central_differences():
    x, w, dy = _case()

    def loss(x, w):
        return np.nansum(grouped_mm(x, w, OFF) * dy)

    dx, dw = grouped_mm_grad_input(dy, w, OFF), grouped_mm_grad_weight(dy, x, OFF)
    h = 1e-5
    for a, da in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + h
            up = loss(x, w)
            a[i] = old - h
            num = (up - loss(x, w)) / (2 * h)
            a[i] = old
            assert abs(num - np.nan_to_num(da[i])) < 1e-8
    assert not dw[1].any()
