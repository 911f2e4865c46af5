"""The rounding model of the orthogonalisation against the stated accuracy, whatever the
rank of the matrix: roundings along directions with singular value zero must not grow."""

import numpy as np
import pytest

from muon_matrices import distance, matrices, stated
from oracle import muon as OM


@pytest.mark.parametrize("shape", [(2, 3), (8, 1000), (16, 16), (16, 24), (32, 1024), (64, 128), (64, 768), (128, 256), (200, 330),
                                   (320, 512), (300, 700), (512, 512)])
def test_stated_accuracy(shape):
    for name, x in matrices(*shape):
        e = OM.orthogonalize(x)
        d = distance(OM.orthogonalize_f16(x, plan=OM.plan(*shape)), e)
        assert d <= stated(*shape), (shape, name, d)


@pytest.mark.parametrize("shape", [(16, 24), (64, 256), (96, 96), (300, 500)])
def test_more_steps(shape):
    """Eight steps of the usual coefficients multiply a rounding along a direction with
    singular value zero by 3.4^7 = 5,800: 2^-12 of an entry would become more than the entry."""
    for name, x in matrices(*shape, seed=1):
        e = OM.orthogonalize(x, steps=8)
        d = distance(OM.orthogonalize_f16(x, steps=8, plan=OM.plan(*shape, 8)), e)
        assert d <= stated(*shape, 8), (shape, name, d)


def test_what_is_left_out_by_hand():
    """A matrix of rank 1 whose FP16 rest lies along no direction of the polynomial but a I:
    one phase of three steps (not among the last two) keeps the rest times a exactly."""
    S, LO = 1024.0, 2048.0
    half = lambda v: np.float64(np.float16(np.float32(v)))
    x = np.array([[1.0, 0.0], [0.0, 2.0 ** -9]])             # entry (1, 1) after scaling has a rest
    t = x / (np.sqrt((x * x).sum()) + 1e-7)
    hi = half(t[1, 1] * S) / S
    lo = half((t[1, 1] - hi) * S * LO) / (S * LO)
    coefs = [(3.0, -1.0, 0.5), (1.0, 0.0, 0.0), (1.0, 0.0, 0.0)]   # the last two phases change nothing
    got = OM.orthogonalize_f16(x, steps=3, coefs=coefs)[1, 1]
    a, b, c = coefs[0]
    p = np.float64(np.float32(a + b * np.float32(hi * hi) + c * np.float64(np.float32(hi * hi)) ** 2))
    assert abs(got - (p * hi + a * lo)) <= 2.0 ** -21 * abs(got)
