"""Pins of the oracles of the 8-bit integer and the orthogonalised-update operators."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import int8 as OI
from oracle import muon as OM


def _rne(v):
    """Nearest integer of a Fraction, ties to even."""
    f = v.numerator // v.denominator
    d = v - f
    return f + (1 if d > Fraction(1, 2) or (d == Fraction(1, 2) and f % 2) else 0)


def _f32(v):
    """A Fraction rounded to FP32 (normal range) by integer arithmetic."""
    if v == 0:
        return Fraction(0)
    s, v = (1, v) if v > 0 else (-1, -v)
    e = 0
    while v >= 2:
        v, e = v / 2, e + 1
    while v < 1:
        v, e = v * 2, e - 1
    return s * Fraction(_rne(v * (1 << 23)), 1 << 23) * Fraction(2) ** e


def test_quantize_by_fractions():
    rng = np.random.RandomState(0)
    x = (rng.randn(7, 33) * np.exp(rng.randn(7, 1))).astype(np.float32)
    x[3] = 0
    bits = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
    codes, scales = OI.quantize(bits)
    vals = (bits.astype(np.uint32) << 16).view(np.float32)
    for r in range(7):
        amax = max(abs(Fraction(float(v))) for v in vals[r])
        enc = Fraction(1) if amax == 0 else _f32(127 * _f32(1 / amax))
        assert Fraction(float(scales[r])) == _f32(1 / enc)
        assert [_rne(_f32(Fraction(float(v)) * enc)) for v in vals[r]] == [int(c) for c in codes[r]]
        assert amax == 0 or np.abs(codes[r].astype(int)).max() == 127


def test_quantize_extremes():
    f = np.float32
    x = np.array([[f(2.0) ** -133, 0, -f(2.0) ** -133, f(2.0) ** -134 * 0],        # subnormal: the scale is clamped
                  [3e38, -1e38, 1e-38, 0], [0, 0, 0, 0]], dtype=np.float32)
    bits = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
    codes, scales = OI.quantize(bits)
    assert np.isfinite(scales).all() and (scales > 0).all() and scales[2] == 1
    assert codes[0].tolist() == [0, 0, 0, 0]                  # 2^-133 times the largest scale, 2^128, rounds to 0
    assert codes[1].tolist()[0] == 127 and codes[1].tolist()[2:] == [0, 0]


def test_gemm_by_integers():
    rng = np.random.RandomState(1)
    a, b = rng.randint(-127, 128, (5, 40)).astype(np.int8), rng.randint(-127, 128, (6, 40)).astype(np.int8)
    sa, sb = rng.rand(5).astype(np.float32), rng.rand(6).astype(np.float32)
    bias = rng.randn(6).astype(np.float32)
    got = OI.gemm(a, sa, b, sb, bias)
    for i in range(5):
        for j in range(6):
            s = sum(int(x) * int(y) for x, y in zip(a[i], b[j]))
            y = np.float32(np.float32(s) * np.float32(sa[i] * sb[j])) + bias[j]
            assert got[i, j] == float(torch.tensor(float(y)).bfloat16())


@pytest.mark.parametrize("shape", [(6, 6), (5, 17), (17, 5), (1, 9)])
def test_orthogonalize_acts_on_singular_values(shape):
    """The polynomial of each step, applied to the singular values by numbers."""
    rng = np.random.RandomState(2)
    x = rng.randn(*shape)
    u, s, vt = np.linalg.svd(x, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    for _ in range(5):
        s = OM.COEFS[0] * s + OM.COEFS[1] * s ** 3 + OM.COEFS[2] * s ** 5
    assert np.allclose(OM.orthogonalize(x), (u * s) @ vt, atol=1e-12)


def test_orthogonalize_converges_with_classical_coefficients():
    rng = np.random.RandomState(3)
    x = rng.randn(8, 20)
    o = OM.orthogonalize(x, steps=32, coefs=(1.5, -0.5, 0.0))
    assert np.allclose(o @ o.T, np.eye(8), atol=1e-9)
    u, _, vt = np.linalg.svd(x, full_matrices=False)
    assert np.allclose(o, u @ vt, atol=1e-9)


def test_orthogonalize_zero_and_steps():
    assert (OM.orthogonalize(np.zeros((3, 4))) == 0).all()
    two = OM.orthogonalize(np.eye(4), steps=2, coefs=[(2.0, -1.5, 0.5), (1.5, -0.5, 0.0)])
    s = 0.5
    s = 2.0 * s - 1.5 * s ** 3 + 0.5 * s ** 5
    s = 1.5 * s - 0.5 * s ** 3
    assert np.allclose(two, s * np.eye(4), atol=1e-6)


def test_f16_form_and_phases():
    """The form with FP16 products stays near the definition for every plan, and is exact
    where nothing rounds."""
    rng = np.random.RandomState(4)
    x = rng.randn(40, 100)
    e = OM.orthogonalize(x)
    for plan in ([1] * 5, [2, 1, 2]):
        f = OM.orthogonalize_f16(x, plan=plan)
        assert 0 < np.linalg.norm(f - e) < 2.0 ** -11 * 5 * np.linalg.norm(e)
    assert np.allclose(OM.orthogonalize_f16(2.0 * np.eye(4), steps=1, coefs=(1.0, 0.0, 0.0), eps=1e-30), 0.5 * np.eye(4))
    assert OM.phases(320, 320, 5) == OM.phases(256, 512, 5) == [1] * 5 and OM.phases(320, 640, 5) == [2, 1, 2]
    assert OM.phases(320, 640, 3, [(8.3, 0, 0), (4.1, 0, 0), (2.9, 0, 0)]) == [1, 2]
    assert OM.phases(320, 640, 7, (1.5, -0.5, 0)) == [2, 1, 2, 1, 1]
    assert OM.plan(64, 128) == OM.plan(512, 96) == OM.plan(512, 97) == [1] * 5 and OM.plan(520, 1000) == [2, 1, 2]


def test_moment():
    m, u = OM.moment(np.float32(2), np.float32(0.5), 0.95, True)
    assert m == np.float32(np.float32(0.95) * np.float32(2)) + np.float32(0.5)
    assert u == np.float32(0.5) + np.float32(np.float32(0.95) * m)
    assert OM.moment(np.float32(2), np.float32(0.5), 0.95, False)[1] == m
