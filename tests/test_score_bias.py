"""Selection by score + bias: the oracle's pins and the entry point's refusals (no GPU)."""

import os

import numpy as np
import pytest

import fp8_quantized_gemm_amd as bsq
from oracle import moe as OM


def test_select_by_score_is_not_select_by_logit():
    """By hand: sigmoid(6, 4, 0) = .9975, .9820, .5; softmax = .8788, .1189, .0022."""
    l = np.array([[6, 4, 0]], np.float32)
    up = np.array([0, 0.02, 0], np.float32)
    assert OM.select(l, up, 1).tolist() == [[0]]                       # 6 > 4.02
    assert OM.select_by_score(l, up, 1, "sigmoid").tolist() == [[1]]   # 1.0020 > .9975
    assert OM.select_by_score(l, up, 1, "softmax").tolist() == [[0]]   # .8788 > .1389
    big = np.array([0, 0, 0.9], np.float32)
    assert OM.select(l, big, 2).tolist() == [[0, 1]]
    assert OM.select_by_score(l, big, 2, "softmax").tolist() == [[2, 0]]
    zero = np.zeros(3, np.float32)
    for scoring in ("sigmoid", "softmax"):                             # without a bias the order is the logits'
        assert OM.select_by_score(l, zero, 3, scoring).tolist() == [[0, 1, 2]]


def test_select_by_score_masks_and_ties():
    inf = np.inf
    l = np.array([[-inf, 0, 0, np.nan], [-inf] * 4, [1, 1, 1, 1]], np.float32)
    b = np.array([5, 0, 0, 5], np.float32)
    for scoring in ("sigmoid", "softmax"):
        assert OM.select_by_score(l, b, 3, scoring).tolist() == [[1, 2, -1], [-1, -1, -1], [0, 3, 1]]
        masked = np.array([0, -inf, np.nan, 0], np.float32)
        assert OM.select_by_score(l, masked, 3, scoring).tolist() == [[-1] * 3, [-1] * 3, [0, 3, -1]]


@pytest.mark.skipif(not os.path.exists(bsq.LIB_PATH), reason="libbsq.so not built (run __graft_entry__.build())")
def test_refusals():
    A, B, C, D, E, F, G = (0x1000000 * i for i in range(1, 8))
    def f(lg=A, T=16, E_=8, k=2, bias=B, sc=0, rows=32, ids=C, w=D, off=E, ro=F, src=G):
        return bsq.lib().moe_route_score_bias(lg, 0, T, E_, k, bias, sc, 1, 1.0, 1, rows, ids, w, off, ro, src, None, 0, None)
    assert f(bias=None) == bsq.BSQ_EINVAL and f(bias=B + 2) == bsq.BSQ_EINVAL
    assert f(k=9) == bsq.BSQ_EINVAL and f(E_=513) == bsq.BSQ_EUNSUPPORTED and f(sc=2) == bsq.BSQ_EINVAL
    assert f(rows=31) == bsq.BSQ_EINVAL and f(lg=None) == bsq.BSQ_EINVAL and f(src=None) == bsq.BSQ_EINVAL
    assert f(T=128, rows=256) == bsq.BSQ_EINVAL                        # no workspace
