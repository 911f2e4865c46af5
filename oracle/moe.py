"""Expert routing and expert-grouped products, plain and slow.

Test infrastructure only (see oracle/__init__.py).  The source pages name no
formulas for a mixture-of-experts layer; the definitions are those include/bsq.h
writes out.  Selection is exact (FP32 logit + bias, or the rounded score +
score_bias; ties to the lowest expert);
weights, gradients and products are float64.
"""

import numpy as np


def rows_bound(tokens, experts, k, align):
    n = tokens * k
    return n if align == 1 else -(-(n + min(experts, n) * (align - 1)) // 512) * 512


def select(logits, bias, k):
    """experts [T, k] (-1: none left) of float32 logits."""
    T, E = logits.shape
    out = np.full((T, k), -1, np.int64)
    with np.errstate(invalid="ignore"):
        score = logits.astype(np.float32) + (0 if bias is None else bias.astype(np.float32))
    for t in range(T):
        left = [e for e in range(E) if logits[t, e] > -np.inf and score[t, e] > -np.inf]
        for j in range(k):
            if not left:
                break
            best = max(left, key=lambda e: (score[t, e], -e))
            out[t, j] = best
            left.remove(best)
    return out


def scores(logits, scoring):
    """float64 scores [T, E] of the logits that are not masked (0 for the others)."""
    l = logits.astype(np.float64)
    ok = l > -np.inf
    if scoring == "sigmoid":
        return np.where(ok, _sigmoid(np.where(ok, l, 0)), 0)
    z = np.where(ok, np.exp(np.where(ok, l, -np.inf) - np.max(np.where(ok, l, -1e300), axis=1, keepdims=True)), 0)
    return z / np.maximum(z.sum(1, keepdims=True), 1e-300)


def select_by_score(logits, score_bias, k, scoring):
    """experts [T, k] by FP32 score + score_bias."""
    s = scores(logits, scoring).astype(np.float32)
    return select(np.where(logits > -np.inf, s, np.float32(-np.inf)), score_bias, k)


def _sigmoid(l):
    return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))


def probabilities(l, ids, scoring, normalize):
    """p over one token's experts [E] (0 where not selected or masked), float64."""
    l = l.astype(np.float64)
    E = len(l)
    sel = np.zeros(E, bool)
    sel[ids[ids >= 0]] = True
    ok = l > -np.inf
    p = np.zeros(E)
    if not sel.any():
        return p
    if scoring == "sigmoid":
        if normalize:
            ls = np.minimum(l[sel], 0) - np.log1p(np.exp(-np.abs(l[sel])))
            z = np.exp(ls - ls.max())
            p[sel] = z / z.sum()
        else:
            p[sel] = _sigmoid(l[sel])
        return p
    over = sel if normalize else ok
    z = np.exp(l[over] - l[over].max())
    p[over] = z / z.sum()
    p[~sel] = 0
    return p


def route(logits, k, bias=None, scoring="softmax", normalize=True, scale=1.0, align=1, score_bias=None):
    T, E = logits.shape
    ids = select(logits, bias, k) if score_bias is None else select_by_score(logits, score_bias, k, scoring)
    w = np.zeros((T, k))
    for t in range(T):
        p = probabilities(logits[t], ids[t], scoring, normalize)
        w[t] = np.where(ids[t] >= 0, scale * p[np.maximum(ids[t], 0)], 0)
    return dict(experts=ids, weights=w, **plan(ids, E, align, rows_bound(T, E, k, align)))


def plan(ids, E, align, rows):
    T, k = ids.shape
    groups = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                groups[ids[t, j]].append(t * k + j)
    off, row_of, src = np.zeros(E + 1, np.int64), np.full(T * k, -1, np.int64), np.full(rows, -1, np.int64)
    for e, g in enumerate(groups):
        for i, a in enumerate(g):
            row_of[a] = off[e] + i
            src[off[e] + i] = a
        off[e + 1] = off[e] + -(-len(g) // align) * align
    return dict(offsets=off, row_of=row_of.reshape(T, k), src=src)


def route_backward(logits, ids, d_w, scoring="softmax", normalize=True, scale=1.0):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        sel = ids[t][ids[t] >= 0]
        if len(sel) == 0:
            continue
        l = logits[t].astype(np.float64)
        g = np.zeros(E)
        g[sel] = scale * d_w[t][ids[t] >= 0]
        p = probabilities(logits[t], ids[t], scoring, normalize)
        if scoring == "sigmoid" and not normalize:
            out[t, sel] = (g * p * _sigmoid(-l))[sel]
        elif scoring == "sigmoid":
            out[t, sel] = (p * (g - (p * g).sum()) * _sigmoid(-l))[sel]
        elif normalize:
            out[t] = p * (g - (p * g).sum())
        else:
            ok = l > -np.inf
            full = np.zeros(E)
            full[ok] = np.exp(l[ok] - l[ok].max())
            full /= full.sum()
            out[t] = full * (g - (p * g).sum())
    return out


def gather(x, src, k):
    out = np.zeros((len(src), x.shape[1]))
    for p, a in enumerate(src):
        if 0 <= a < len(x) * k:
            out[p] = x[a // k]
    return out


def combine(y, row_of, w=None):
    T, k = row_of.shape
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= row_of[t, j] < len(y):
                out[t] += (1.0 if w is None else w[t, j]) * y[row_of[t, j]]
    return out


def combine_backward(d_out, y, src, row_of, w):
    T, k = row_of.shape
    d_y, d_w = np.zeros_like(y), np.zeros((T, k))
    for p, a in enumerate(src):
        if 0 <= a < T * k:
            d_y[p] = w.reshape(-1)[a] * d_out[a // k]
            if row_of[a // k, a % k] == p:
                d_w[a // k, a % k] = d_out[a // k] @ y[p]
    return d_y, d_w


def grouped(a, b, offsets):
    """[rows, N] of dequantized a [rows, K], b [E, N, K], and the sums of absolute products."""
    out, mag = np.zeros((len(a), b.shape[1])), np.zeros((len(a), b.shape[1]))
    for e in range(len(b)):
        s = slice(offsets[e], offsets[e + 1])
        out[s], mag[s] = a[s] @ b[e].T, np.abs(a[s]) @ np.abs(b[e]).T
    return out, mag


def grouped_wgrad(a, b, offsets):
    """[E, M, N] of dequantized a [M, rows], b [N, rows], and the sums of absolute products."""
    E = len(offsets) - 1
    out, mag = np.zeros((E, len(a), len(b))), np.zeros((E, len(a), len(b)))
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        out[e], mag[e] = a[:, s] @ b[:, s].T, np.abs(a[:, s]) @ np.abs(b[:, s]).T
    return out, mag
