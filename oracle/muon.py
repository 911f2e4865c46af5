"""Newton-Schulz orthogonalisation and the weight update that takes it (definitions in
include/bsq.h).

orthogonalize: the definition in FP64.  orthogonalize_f16: the same with what is held
between products rounded to FP16 as the kernels hold it, for the size of error that
these roundings cause; sums are FP64 here, FP32 in the kernels."""

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
    """Numbers of steps that are taken on one Gram matrix, in turn: one by one on
    nearly square matrices; else up to three while the product of the leading
    coefficients is at most 48."""
    lead = [abs(float(v[0])) for v in _steps(steps, coefs)]
    out, i = [], 0
    while i < steps:
        r, p = 1, lead[i]
        while 2 * n >= 3 * m and r < 3 and i + r < steps and p * lead[i + r] <= 48:
            p *= lead[i + r]
            r += 1
        out.append(r)
        i += r
    return out


def orthogonalize_f16(x, steps=5, coefs=COEFS, eps=1e-7, plan=None):
    def half(v, scale):
        return (v * scale).astype(np.float32).astype(np.float16).astype(np.float64) / scale

    def mirror(v):
        return np.tril(v) + np.tril(v, -1).T
    X, A, P = 1024.0, 1024.0, 256.0
    x = np.asarray(x, dtype=np.float64)
    t = _small_side(x)
    t = half(t / (np.sqrt((t * t).sum()) + eps), X)
    eye, c = np.eye(t.shape[0]), _steps(steps, coefs)
    plan = [1] * steps if plan is None else plan
    i = 0
    for k, r in enumerate(plan):
        g, p = half(mirror(t @ t.T), A), None
        for j in range(r):
            q = half(mirror(c[i][0] * eye + c[i][1] * g + c[i][2] * (g @ g)), P)
            if j + 1 < r:
                g = half(mirror(half(mirror(q @ g), A) @ q), A)
            p = q if p is None else half(mirror(q @ p), P)
            i += 1
        t = p @ t
        if k + 1 < len(plan):
            t = half(t, X)
    return t.T if x.shape[0] > x.shape[1] else t


def moment(momentum, grad, mu, nesterov):
    """(new momentum, what is orthogonalised), FP32 with a rounding after each operation."""
    f = np.float32
    m = (f(mu) * momentum).astype(f) + grad
    return m, (grad + (f(mu) * m).astype(f)) if nesterov else m
