"""Edges of the norm, the router and the row movers."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from oracle import moe as OM

from _gpu import announce, gpu

pytestmark = gpu

U = 2.0 ** -24


def _np(t):
    return t.detach().double().cpu().numpy()


def _combine_backward(d, y, src, row_of, w):
    """Through the C entry with the outputs full of NaN."""
    (T, k), (R, C) = row_of.shape, y.shape
    d_y, d_w = torch.full_like(y, float("nan")), torch.full_like(w, float("nan"))
    p = lambda t: t.data_ptr()
    st = bsq.lib().moe_combine_backward(p(d), p(y), T, C, k, p(src), p(row_of), p(w), R, p(d_y), p(d_w),
                                        torch.cuda.current_stream().cuda_stream)
    assert st == bsq.BSQ_OK
    return d_y, d_w


@pytest.mark.parametrize("T,C", [(3, 64), (300, 520), (5, 7)])
@pytest.mark.parametrize("what", ["cut", "slots", "rows"])
def test_combine_backward_of_slots_without_a_row(T, C, what):
    """d_weights of a slot that combine left out, or whose row is not its own, is 0:
    the expert buffer cut to a capacity, slots taken out of row_of, rows out of src."""
    announce("moe_combine_backward without rows", T, C, what)
    g = torch.Generator(device="cuda").manual_seed(T + C)
    k = 2
    f = bsq.moe_route(torch.randn((T, 4), generator=g, device="cuda"), k, align=16)
    src, row_of, w = f["src"].clone(), f["row_of"].clone(), f["weights"]
    if what == "cut":
        src = src[:(2 * T + 1) // 3].contiguous()
    elif what == "slots":
        row_of[::2, 1] = -1
        row_of[1, 0] = 1 << 30
    else:
        src[::3] = -1
    y = torch.randn((len(src), C), generator=g, device="cuda").bfloat16()
    d = torch.randn((T, C), generator=g, device="cuda").bfloat16()
    d_y, d_w = _combine_backward(d, y, src, row_of, w)
    sn, rn = src.cpu().numpy(), row_of.cpu().numpy()
    wy, ww = OM.combine_backward(_np(d), _np(y), sn, rn, _np(w))
    _, mag = OM.combine_backward(np.abs(_np(d)), np.abs(_np(y)), sn, rn, np.ones((T, k)))
    own = np.zeros((T, k), bool)
    for t in range(T):
        for j in range(k):
            r = rn[t, j]
            own[t, j] = 0 <= r < len(sn) and sn[r] == t * k + j
    assert not own.all()
    assert not ww[~own].any() and not mag[~own].any()
    assert np.all(np.abs(_np(d_w) - ww) <= (C / 64 + 16) * U * mag)       # 0 exactly where there is no row
    assert np.all(np.abs(_np(d_y) - wy) <= 2.0 ** -8 * np.abs(wy) + 2 * U * np.abs(wy))
    for _ in range(3):
        again = _combine_backward(d, y, src, row_of, w)
        assert torch.equal(again[0], d_y) and torch.equal(again[1], d_w)
