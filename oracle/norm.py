"""Norms around a block with its gate and residual scale, and their gradient.

Test infrastructure only (see oracle/__init__.py).  The source pages give no
formulas for these parts of the transformer layer; the usual definitions are
taken (root-mean-square norm, a gate on the block's output, a scaled residual),
evaluated in float64 on the inputs as stored:

    n = o * rstd_post * w_post,  r = alpha * x + gate * n,  h = r * rstd_pre * w_pre
    rstd(v) = (mean over the row of v^2 + eps)^(-1/2)
"""

import numpy as np


def rstd(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1) + eps)


def forward(x, o=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=1e-6):
    """dict(r, h, rstd_post, rstd_pre); entries that do not apply are None."""
    r, rq, n = x, None, o
    if o is not None:
        if w_post is not None:
            rq = rstd(o, eps)
            n = o * rq[:, None] * w_post
        r = alpha * x + (n if gate is None else gate * n)
    h = rp = None
    if w_pre is not None:
        rp = rstd(r, eps)
        h = r * rp[:, None] * w_pre
    return dict(r=r if o is not None else None, h=h, rstd_post=rq, rstd_pre=rp)


def backward(r, o=None, d_r=None, d_h=None, w_pre=None, w_post=None, gate=None, rstd_pre=None,
             rstd_post=None, alpha=1.0):
    """dict(d_x, d_o, d_gate, d_w_pre, d_w_post) with r, o and the rstd given, plus
    the sums of absolute terms of each (keys with a trailing underscore), the
    scale of its rounding errors."""
    out = {}
    G = np.zeros_like(r) if d_r is None else d_r.astype(np.float64)
    Gm = np.abs(G)
    if w_pre is not None:
        rn, a = r * rstd_pre[:, None], d_h * w_pre
        mean = np.mean(a * rn, axis=1, keepdims=True)
        G = G + rstd_pre[:, None] * (a - rn * mean)
        Gm = Gm + rstd_pre[:, None] * (np.abs(a) + np.abs(rn) * np.mean(np.abs(a * rn), axis=1, keepdims=True))
        out["d_w_pre"], out["d_w_pre_"] = (d_h * rn).sum(0), np.abs(d_h * rn).sum(0)
    out["d_x"], out["d_x_"] = (G if o is None else alpha * G), Gm * (1.0 if o is None else abs(alpha))
    if o is None:
        return out
    on = o if w_post is None else o * rstd_post[:, None]
    n = on if w_post is None else on * w_post
    g = 1.0 if gate is None else gate
    if gate is not None:
        t, tm = G * n, Gm * np.abs(n)
        if gate.ndim == 1:
            t, tm = t.sum(0), tm.sum(0)
        elif gate.shape[1] == 1 and r.shape[1] != 1:
            t, tm = t.sum(1, keepdims=True), tm.sum(1, keepdims=True)
        out["d_gate"], out["d_gate_"] = t, tm
    if w_post is None:
        out["d_o"], out["d_o_"] = G * g * np.ones_like(o), Gm * np.abs(g) * np.ones_like(o)
        return out
    b, bm = G * g * w_post, Gm * np.abs(g * w_post)
    k = rstd_post[:, None]
    out["d_o"] = k * (b - on * np.mean(b * on, axis=1, keepdims=True))
    out["d_o_"] = k * (bm + np.abs(on) * np.mean(bm * np.abs(on), axis=1, keepdims=True))
    out["d_w_post"], out["d_w_post_"] = (G * g * on).sum(0), (Gm * np.abs(g * on)).sum(0)
    return out
