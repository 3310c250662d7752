"""Orthogonalised updates in 64 bits: Newton-Schulz steps on one matrix."""

import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def start(g):
    g = np.asarray(g, np.float64)
    norm = np.sqrt((g * g).sum())
    return g / norm if norm > 0 else g


def step(x, abc):
    a, b, c = abc
    m = x @ x.T
    return a * x + (b * m + c * (m @ m)) @ x


def orthogonalize(g, steps=5, coefficients=COEFFICIENTS):
    x = start(g)
    for _ in range(steps):
        x = step(x, coefficients)
    return x
