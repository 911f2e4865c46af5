"""Newton-Schulz orthogonalisation and the weight update that takes it (definitions in
include/bsq.h).

orthogonalize: the definition in FP64.  orthogonalize_f16: the same with what is held
between products rounded as the kernels hold it (X as an FP16 matrix and the FP16 rest
of its rounding, symmetric matrices as an FP32 diagonal and an FP16 rest), for the size
of error that these roundings cause; sums are FP64 here, FP32 in the kernels.

The rest of X's rounding is multiplied by the phase's leading coefficient (the product of a
pair's), in the last two phases by the polynomial's diagonal, in place of the polynomial
P = a I + b A + c A^2.  What that leaves out, (P - a) lo, is zero on directions with singular
value zero, the only ones along which it would grow (by a in each step that follows)."""

import numpy as np

COEFS = (3.4445, -4.7750, 2.0315)


def _steps(steps, coefs):
    c = np.asarray(coefs, dtype=np.float64)
    return np.broadcast_to(c, (steps, 3)) if c.ndim == 1 else c


def _small_side(x):
    return x.T if x.shape[0] > x.shape[1] else x


def orthogonalize(x, steps=5, coefs=COEFS, eps=1e-7):
    x = np.asarray(x, dtype=np.float64)
    t = _small_side(x)
    t = t / (np.sqrt((t * t).sum()) + eps)
    for a, b, c in _steps(steps, coefs):
        g = t @ t.T
        t = a * t + (b * g + c * (g @ g)) @ t
    return t.T if x.shape[0] > x.shape[1] else t


def phases(m, n, steps, coefs=COEFS):
    """Numbers of steps that are taken on one Gram matrix, in turn: one by one, or, from
    n = 4/3 m on and m above 256, pairs with a single step between them, of steps whose leading
    coefficients' product is at most 12."""
    lead = [abs(float(np.float32(v[0]))) for v in _steps(steps, coefs)]
    out = []
    while sum(out) < steps:
        i = sum(out)
        pair = m > 256 and 3 * n >= 4 * m and out[-1:] != [2] and i + 2 <= steps and lead[i] * lead[i + 1] <= 12
        out.append(2 if pair else 1)
    return out


def plan(rows, cols, steps=5, coefs=COEFS):
    """The phases that orthogonalize takes: single steps where one workgroup holds the
    matrix, else those of the sizes padded to 64."""
    m, n = sorted((rows, cols))
    up = lambda v, k: (v + k - 1) // k * k
    a, b = up(m, 32), up(n, 32)
    lds = a * (a + 8) * 2 + a * 4 + 2 * max(a * (b + 8), b * (a + 8))
    if m <= 160 and n <= (1024 if m <= 32 else 768 if m <= 64 else 512 if m <= 96 else 256) and lds + 64 <= 160 * 1024:
        return [1] * steps
    return phases(up(m, 64), up(n, 64), steps, coefs)


def orthogonalize_f16(x, steps=5, coefs=COEFS, eps=1e-7, plan=None):
    S, LO = 1024.0, 2048.0

    def half(v):
        return v.astype(np.float32).astype(np.float16).astype(np.float64)

    def split(v):
        """A symmetric matrix as (diagonal, FP16 rest)."""
        v = np.tril(v) + np.tril(v, -1).T
        return np.diag(v).astype(np.float32).astype(np.float64), half((v - np.diag(np.diag(v))) * S) / S

    def times(l, r):
        return l[1] @ r[1] + l[0][:, None] * r[1] + l[1] * r[0][None, :] + np.diag(l[0] * r[0])
    x = np.asarray(x, dtype=np.float64)
    t = _small_side(x)
    t = t / (np.sqrt((t * t).sum()) + eps)
    eye, c = np.eye(t.shape[0]), _steps(steps, coefs)
    plan = [1] * steps if plan is None else plan
    i = 0
    for phase, r in enumerate(plan):
        hi = half(t * S) / S
        lo = half((t - hi) * S * LO) / (S * LO)
        lead = np.prod([c[i + j][0] for j in range(r)])
        g, p = split(hi @ hi.T), None
        for j in range(r):
            q = split(c[i][0] * eye + c[i][1] * (np.diag(g[0]) + g[1]) + c[i][2] * times(g, g))
            if j + 1 < r:
                g = split(times(split(times(q, g)), q))
            p = q if p is None else split(times(q, p))
            i += 1
        t = p[0][:, None] * hi + (lead if phase + 2 < len(plan) else p[0][:, None]) * lo + p[1] @ hi
    return t.T if x.shape[0] > x.shape[1] else t


def moment(momentum, grad, mu, nesterov):
    """(new momentum, what is orthogonalised), FP32 with a rounding after each operation."""
    f = np.float32
    m = (f(mu) * momentum).astype(f) + grad
    return m, (grad + (f(mu) * m).astype(f)) if nesterov else m
