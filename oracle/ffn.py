"""The experts' gated feed-forward block over rows sorted by expert, and its
gradients, in 64 bits: out = down (silu(g) * u), (g, u) = gate_up x."""

import numpy as np


def sigmoid(g):
    g = np.asarray(g, np.float64)
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + e), e / (1 + e))


def _spans(offsets, E):
    return [(e, slice(int(offsets[e]), int(offsets[e + 1]))) for e in range(E)]


def pre_activations(x, gate_up, offsets):
    """[M, H], [E, 2I, H] -> g | u [M, 2I]; NaN where no expert owns the row."""
    gu = np.full((x.shape[0], gate_up.shape[1]), np.nan)
    for e, p in _spans(offsets, gate_up.shape[0]):
        gu[p] = np.asarray(x[p], np.float64) @ np.asarray(gate_up[e], np.float64).T
    return gu


def hidden(gu):
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    return g * sigmoid(g) * u


def ffn(x, gate_up, down, offsets):
    """-> out [M, H]; NaN where no expert owns the row."""
    h = hidden(pre_activations(x, gate_up, offsets))
    out = np.full((x.shape[0], down.shape[1]), np.nan)
    for e, p in _spans(offsets, down.shape[0]):
        out[p] = h[p] @ np.asarray(down[e], np.float64).T
    return out


def activation_gradients(dh, gu):
    """dL/dh [M, I], g | u [M, 2I] -> dL/d(g | u) [M, 2I]."""
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    s = sigmoid(g)
    return np.concatenate([dh * u * s * (1 + g * (1 - s)), dh * g * s], axis=1)


def ffn_backward(dy, x, gate_up, down, offsets, gu):
    """-> (grad_x [M, H], grad_gate_up [E, 2I, H], grad_down [E, H, I]), from
    the pre-activations gu [M, 2I]."""
    dx = np.full(np.shape(x), np.nan)
    dw1, dw2 = np.zeros(gate_up.shape), np.zeros(down.shape)
    h = hidden(gu)
    for e, p in _spans(offsets, down.shape[0]):
        d, xe = np.asarray(dy[p], np.float64), np.asarray(x[p], np.float64)
        dgu = activation_gradients(d @ np.asarray(down[e], np.float64), gu[p])
        dx[p] = dgu @ np.asarray(gate_up[e], np.float64)
        dw1[e], dw2[e] = dgu.T @ xe, d.T @ h[p]
    return dx, dw1, dw2
