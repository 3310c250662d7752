"""Products grouped by expert in 64 bits, over rows sorted by expert: rows
offsets[e] <= p < offsets[e+1] belong to expert e."""

import numpy as np


def grouped_mm(x, w, offsets):
    """[M, K], [E, N, K] -> [M, N]; NaN where no expert owns the row."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        y[lo:hi] = np.asarray(x[lo:hi], np.float64) @ np.asarray(w[e], np.float64).T
    return y


def grouped_mm_grad_input(dy, w, offsets):
    """[M, N], [E, N, K] -> [M, K]; NaN where no expert owns the row."""
    dx = np.full((dy.shape[0], w.shape[2]), np.nan)
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        dx[lo:hi] = np.asarray(dy[lo:hi], np.float64) @ np.asarray(w[e], np.float64)
    return dx


def grouped_mm_grad_weight(dy, x, offsets):
    """[M, N], [M, K] -> [E, N, K]."""
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        dw[e] = np.asarray(dy[lo:hi], np.float64).T @ np.asarray(x[lo:hi], np.float64)
    return dw
