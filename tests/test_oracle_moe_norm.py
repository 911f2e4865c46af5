"""Pins of the oracle's norm, router and grouped-product references (no GPU):
gradients against central differences, closed forms, and brute force."""

import numpy as np
import pytest

from oracle import moe as OM
from oracle import norm as ON


def _diff(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + h
        up = f()
        x[i] = old - h
        g[i] = (up - f()) / (2 * h)
        x[i] = old
    return g


NORMS = [(g,) + f for g in (None, "channel", "row", "full") for f in ((1, 1, 1), (1, 0, 1), (1, 1, 0))]


@pytest.mark.parametrize("gate,has_o,post,pre", NORMS + [(None, 0, 0, 1)])
def test_norm_gradient_is_the_difference_quotient(gate, has_o, post, pre):
    rng = np.random.default_rng(3)
    R, C = 3, 5
    x, o = rng.normal(size=(R, C)), rng.normal(size=(R, C)) if has_o else None
    wp = 1 + 0.3 * rng.normal(size=C) if pre else None
    wq = 1 + 0.3 * rng.normal(size=C) if post else None
    g = {None: None, "channel": rng.normal(size=C), "row": rng.normal(size=(R, 1)), "full": rng.normal(size=(R, C))}[gate]
    d_r, d_h = rng.normal(size=(R, C)) if has_o else None, rng.normal(size=(R, C)) if pre else None
    kw = dict(w_pre=wp, w_post=wq, gate=g)

    def loss():
        f = ON.forward(x, o, alpha=0.7, eps=1e-3, **kw)
        return (0 if d_r is None else (f["r"] * d_r).sum()) + (0 if d_h is None else (f["h"] * d_h).sum())
    f = ON.forward(x, o, alpha=0.7, eps=1e-3, **kw)
    b = ON.backward(f["r"] if has_o else x, o, d_r, d_h, rstd_pre=f["rstd_pre"], rstd_post=f["rstd_post"], alpha=0.7, **kw)
    for name, v in (("d_x", x), ("d_o", o), ("d_gate", g), ("d_w_pre", wp), ("d_w_post", wq)):
        if v is not None:
            # second-order differences at 1e-6 in float64: rounding 1e-10, curvature 1e-11
            assert np.allclose(b[name], _diff(loss, v), atol=1e-7), name


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_is_the_difference_quotient(scoring, normalize):
    rng = np.random.default_rng(4)
    T, E, k = 3, 6, 3
    l = rng.normal(size=(T, E)).astype(np.float64)
    l[1, 2] = -np.inf
    l[2, 1:] = -np.inf
    ids, d_w = OM.select(l, None, k), rng.normal(size=(T, k))

    def loss():
        s = 0.0
        for t in range(T):
            p = OM.probabilities(l[t], ids[t], scoring, normalize)
            s += sum(1.5 * p[ids[t, j]] * d_w[t, j] for j in range(k) if ids[t, j] >= 0)
        return s
    got, ok = OM.route_backward(l, ids, d_w, scoring, normalize, 1.5), np.isfinite(l)
    want = np.zeros((T, E))
    for i in np.argwhere(ok):
        i = tuple(i)
        old = l[i]
        l[i] = old + 1e-6
        up = loss()
        l[i] = old - 1e-6
        want[i] = (up - loss()) / 2e-6
        l[i] = old
    assert np.allclose(got, want, atol=1e-7)


def test_select_ties_masks_and_empty_rows():
    l = np.array([[1, 1, 0, 1], [-np.inf, np.nan, -3, -np.inf], [np.nan] * 4, [0.0, -0.0, 0.0, -0.0]], np.float32)
    assert OM.select(l, None, 3).tolist() == [[0, 1, 3], [2, -1, -1], [-1, -1, -1], [0, 1, 2]]
    low = np.full((1, 4), np.finfo(np.float32).min, np.float32)     # the lowest value is a value, not a mask
    assert OM.select(low, None, 2).tolist() == [[0, 1]]
    assert OM.select(np.zeros((1, 3), np.float32), np.array([0, 1, -np.inf], np.float32), 3).tolist() == [[1, 0, -1]]


@pytest.mark.parametrize("align", [1, 16, 32])
def test_plan_is_a_stable_sort(align):
    rng = np.random.default_rng(5)
    T, E, k = 37, 5, 2
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    ids[3] = -1
    ids[7, 1] = -1
    rows = OM.rows_bound(T, E, k, align)
    p = OM.plan(ids, E, align, rows)
    flat = ids.reshape(-1)
    live = np.flatnonzero(flat >= 0)
    order = live[np.argsort(flat[live], kind="stable")]
    assert np.array_equal(p["src"][p["src"] >= 0], order)
    assert np.all(p["offsets"] % align == 0) and p["offsets"][-1] <= rows
    for a in live:
        r = p["row_of"].reshape(-1)[a]
        assert p["src"][r] == a and p["offsets"][flat[a]] <= r < p["offsets"][flat[a] + 1]


def test_combine_is_the_adjoint_of_gather():
    rng = np.random.default_rng(6)
    T, E, k, C = 9, 4, 2, 3
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    ids[2, 0] = -1
    p = OM.plan(ids, E, 4, OM.rows_bound(T, E, k, 4))
    x, z = rng.normal(size=(T, C)), rng.normal(size=(len(p["src"]), C))
    assert np.isclose((OM.gather(x, p["src"], k) * z).sum(), (x * OM.combine(z, p["row_of"])).sum())
    w, d = rng.normal(size=(T, k)), rng.normal(size=(T, C))
    d_y, d_w = OM.combine_backward(d, z, p["src"], p["row_of"], w)
    assert np.allclose(d_y, _diff(lambda: (OM.combine(z, p["row_of"], w) * d).sum(), z), atol=1e-7)
    assert np.allclose(d_w, _diff(lambda: (OM.combine(z, p["row_of"], w) * d).sum(), w), atol=1e-7)


def test_grouped_products_are_the_blocks_of_a_block_diagonal_one():
    rng = np.random.default_rng(7)
    off = [0, 3, 3, 7]
    a, b = rng.normal(size=(9, 4)), rng.normal(size=(3, 5, 4))
    out, mag = OM.grouped(a, b, off)
    for p in range(9):
        e = 0 if p < 3 else 2 if p < 7 else None
        want = np.zeros(5) if e is None else b[e] @ a[p]
        assert np.allclose(out[p], want) and np.all(mag[p] >= np.abs(out[p]) - 1e-12)
    am, bn = rng.normal(size=(2, 9)), rng.normal(size=(3, 9))
    w, _ = OM.grouped_wgrad(am, bn, off)
    assert np.all(w[1] == 0) and np.allclose(w[2], am[:, 3:7] @ bn[:, 3:7].T)
