"""The feed-forward oracle against the closed form at single values, the
per-token loop, and differences."""

import math

import numpy as np

from oracle.ffn import ffn, ffn_backward, hidden, pre_activations, sigmoid

OFF = [1, 3, 3, 6]


def _case(seed=0, M=7, E=3, H=5, I=4):
    r = np.random.default_rng(seed)
    return r.standard_normal((M, H)), r.standard_normal((E, 2 * I, H)), r.standard_normal((E, H, I))


def test_sigmoid_and_hidden():
    for g in (-700.0, -3.0, -0.0, 0.5, 40.0):
        assert math.isclose(float(sigmoid(g)), 1 / (1 + math.exp(-g)), rel_tol=1e-15)
    assert sigmoid(np.array(-1e4)) == 0 and sigmoid(np.array(1e4)) == 1
    h = hidden(np.array([[2.0, -1.0, 3.0, 5.0]]))
    assert np.allclose(h, [[6 / (1 + math.exp(-2)), -5 / (1 + math.exp(1))]], rtol=1e-15)


def test_block_row_by_row():
    x, w1, w2 = _case()
    y = ffn(x, w1, w2, OFF)
    assert np.isnan(y[[0, 6]]).all()
    for e in range(3):
        for p in range(OFF[e], OFF[e + 1]):
            g, u = w1[e, :4] @ x[p], w1[e, 4:] @ x[p]
            assert np.allclose(y[p], w2[e] @ (g / (1 + np.exp(-g)) * u), rtol=1e-13)


def test_gradients_against_differences():
    x, w1, w2 = _case(1)
    dy = np.random.default_rng(2).standard_normal(x.shape)
    grads = ffn_backward(dy, x, w1, w2, OFF, pre_activations(x, w1, OFF))

    def loss():
        return float((ffn(x, w1, w2, OFF)[1:6] * dy[1:6]).sum())

    step = 1e-5
    for t, g in zip((x, w1, w2), grads):
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + step
            up = loss()
            t[i] = keep - step
            down = loss()
            t[i] = keep
            if t is x and i[0] in (0, 6):
                assert np.isnan(g[i]) and up == down
                continue
            # a central difference is off by step^2 / 6 of a third derivative of some hundreds
            assert abs((up - down) / (2 * step) - g[i]) < 1e-6 * max(1.0, abs(g[i])), (i, g[i])
    assert not grads[1][1].any() and not grads[2][1].any()   # an expert without rows
