"""The Newton-Schulz oracle against the polynomial of the singular values."""

import numpy as np

from oracle.orthogonalize import COEFFICIENTS, orthogonalize, start


def test_acts_on_the_singular_values():
    r = np.random.default_rng(0)
    for shape in ((7, 12), (12, 7), (9, 9), (1, 5), (5, 1)):
        g = r.standard_normal(shape)
        u, s, v = np.linalg.svd(start(g), full_matrices=False)
        assert np.isclose((s * s).sum(), 1)
        for _ in range(5):
            s = COEFFICIENTS[0] * s + COEFFICIENTS[1] * s ** 3 + COEFFICIENTS[2] * s ** 5
        assert np.allclose(orthogonalize(g), (u * s) @ v, atol=1e-12)


def test_the_side_does_not_matter_and_zeros_stay():
    g = np.random.default_rng(1).standard_normal((6, 15))
    assert np.allclose(orthogonalize(g), orthogonalize(g.T).T, atol=1e-12)
    assert np.allclose(orthogonalize(g), orthogonalize(1e-30 * g), atol=1e-12)
    assert not orthogonalize(np.zeros((3, 4))).any()
    s = np.linalg.svd(orthogonalize(g), compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.3
