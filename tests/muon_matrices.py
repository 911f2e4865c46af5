"""Matrices on which Newton-Schulz steps in fewer bits go wrong, and the accuracy that
include/bsq.h states for five steps of the usual coefficients (relative, Frobenius)."""

import numpy as np

from oracle import muon as OM


def matrices(m, n, seed=0):
    """(name, matrix [m, n]): full rank, each lower rank, singular values over two and four
    decades, one direction over a small floor, one row."""
    rng = np.random.default_rng(seed)
    k = min(m, n)
    yield "full rank", rng.standard_normal((m, n))
    for r in (1, 2, 8, 32, 64, 128, 256):
        if r < k:
            yield f"rank {r}", rng.standard_normal((m, r)) @ rng.standard_normal((r, n))
    u, v = np.linalg.qr(rng.standard_normal((m, k)))[0], np.linalg.qr(rng.standard_normal((n, k)))[0].T
    for e in (5, 9):
        yield f"singular values over e^{e}", u * np.exp(-e * np.arange(k) / max(1, k - 1)) @ v
    yield "rank 1 over a floor", np.outer(rng.standard_normal(m), rng.standard_normal(n)) + 1e-3 * rng.standard_normal((m, n))
    x = np.zeros((m, n))
    x[m // 2] = rng.standard_normal(n)
    yield "one row", x


def stated(m, n, steps=5):
    """The accuracy of include/bsq.h: five steps 2e-3 one at a time, 5e-3 for fewer than 16
    rows (columns) and in pairs.  Every step rounds as many values to as many bits, and what one
    leaves of FP16's bits does not grow in those after it (along singular values near zero, where
    all would grow, nothing is left; elsewhere the step's polynomial brings singular values
    together), so the roundings of k steps add up to at most k / 5 of those of five.  (The last
    bits of X, 2^-24, do grow: to 2^-24 3.44^8 = 1.2e-3 after eight steps, within the 3.2e-3 that
    this gives for one at a time.  FP32 sums add as much again for each doubling of the square
    root of their length, so smaller sides above 512 are left out for eight steps.)"""
    return (5e-3 if min(m, n) < 16 or 2 in OM.plan(m, n, steps) else 2e-3) * max(1.0, steps / 5)


def distance(x, e):
    return np.linalg.norm(x - e) / np.linalg.norm(e)
