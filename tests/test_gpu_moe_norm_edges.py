"""Edges of the norm, the router and the row movers, and a layer without tokens."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from fp8_quantized_gemm_amd.moe import MoELayer
from oracle import moe as OM
from oracle import norm as ON

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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C", [16, 100, 256, 600, 2048])
@pytest.mark.parametrize("R", [1, 3, 65])
@pytest.mark.parametrize("gate", [None, "channel", "row", "full"])
def test_infinite_gradient_in_the_last_row(R, C, dtype, gate):
    """Column sums are those of the rows there are, an infinite one included: the rows
    that fill up a workgroup's last trip add nothing (not 0 times infinity)."""
    announce("block_norm_backward, infinity in the last row", R, C, dtype, gate)
    g = torch.Generator(device="cuda").manual_seed(R * 3 + C)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, o = rn(R, C).to(dtype), rn(R, C).bfloat16()
    wp, wq = 1 + 0.1 * rn(C), 1 + 0.1 * rn(C)
    gt = {None: None, "channel": 1 + 0.1 * rn(C), "row": 1 + 0.1 * rn(R, 1), "full": (1 + 0.1 * rn(R, C)).bfloat16()}[gate]
    f = bsq.block_norm(x, o, w_pre=wp, w_post=wq, gate=gt)
    d_r, d_h = rn(R, C).to(dtype), rn(R, C).bfloat16()
    d_h[R - 1, 3] = float("inf")
    got = bsq.block_norm_backward(f["r"], o, d_r, d_h, wp, wq, gt, f["rstd_pre"], f["rstd_post"])
    with np.errstate(invalid="ignore"):
        want = ON.backward(_np(f["r"]), _np(o), _np(d_r), _np(d_h), _np(wp), _np(wq), None if gate is None else _np(gt),
                           _np(f["rstd_pre"]), _np(f["rstd_post"]))
    v, w, m = _np(got["d_w_pre"]), want["d_w_pre"], want["d_w_pre_"]
    fine = np.isfinite(w)
    assert fine.sum() == C - 1 and np.isinf(w[3]) and v[3] == w[3]
    assert np.all(np.abs(v[fine] - w[fine]) <= (R + 12) * U * m[fine])          # R additions, 3 roundings a term
    names = ["d_w_post"] + (["d_gate"] if gate == "channel" else [])
    for n in names:                                                       # infinite but for column 3 (inf - inf)
        v, w = _np(got[n]), want[n]
        assert np.isnan(w[3]) and np.isinf(np.delete(w, 3)).all()
        assert np.array_equal(v, w, equal_nan=True), n


def test_layer_without_tokens():
    """A micro-batch of no tokens: empty activations, zero weight gradients."""
    announce("MoELayer without tokens")
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    L = MoELayer(rn(4, 64, 48), rn(4, 48, 32), 2, dict(w_pre=1 + 0.1 * rn(48), w_post=1 + 0.1 * rn(48)))
    x = rn(0, 48).bfloat16()
    L.grad["W_gu"].fill_(3)
    L.grad["W_down"].fill_(3)
    r, h = L.open(x, x)
    y = L.forward(h, rn(0, 4))
    d_h, d_l = L.backward(y)
    grads = L.close(r, d_h)
    assert y.shape == (0, 48) and d_h.shape == (0, 48) and d_l.shape == (0, 4) and r.shape == (0, 48)
    assert not L.grad["W_gu"].any() and not L.grad["W_down"].any()
    assert grads["d_x"].shape == (0, 48) and not grads["d_w_pre"].any() and not grads["d_w_post"].any()
    before = L.w32["W_gu"].clone()
    L.update()
    assert torch.equal(before, L.w32["W_gu"])


@pytest.mark.parametrize("shape", [(0, 64), (64, 0)])
def test_quantizers_of_empty_tensors(shape):
    announce("quantizers of empty tensors", shape)
    x = torch.zeros(shape, device="cuda").bfloat16()
    for fmt in ("nvfp4", "mxfp4", "mxfp8"):
        q = bsq.quantize_transpose(x, fmt)
        assert q["row_codes"].numel() == 0 and q["col_codes"].numel() == 0
    assert not bsq.quantize_transpose(x)["row_amax"].any()
    a = torch.ones(1, device="cuda")
    assert bsq.quantize_transpose_amax(x, a, a)["row_scales"].shape == (shape[0], shape[1] // 16)
    assert not bsq.fp8_quantize_transpose(x)["amax"].any()


@pytest.mark.parametrize("E", [8, 100])
@pytest.mark.parametrize("scoring,normalize", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_an_expert_masked_by_the_bias_keeps_its_share_of_the_full_softmax(E, scoring, normalize):
    """A bias of -inf takes an expert out of the selection and leaves its logit in the
    softmax over all, forward and backward (the selection is constant there)."""
    announce("moe_route, bias of -inf", E, scoring, normalize)
    g = torch.Generator(device="cuda").manual_seed(E)
    T, k = 90, 3
    l, d = torch.randn((T, E), generator=g, device="cuda"), torch.randn((T, k), generator=g, device="cuda")
    l[5, 2:] = float("-inf")                             # what is left is masked by the bias
    b = torch.zeros(E, device="cuda")
    b[:2] = float("-inf")
    f = bsq.moe_route(l, k, b, scoring, normalize)
    got = bsq.moe_route_backward(l, f["experts"], d, scoring, normalize)
    ln = l.cpu().numpy()
    want = OM.route(ln, k, b.cpu().numpy(), scoring, normalize)
    assert np.array_equal(f["experts"].cpu().numpy(), want["experts"]) and (f["experts"] > 1).any()
    assert torch.all(f["experts"][5] == -1) and not f["weights"][5].any() and not got[5].any()
    # the bounds of the router's own tests: 64 roundings of a weight, 128 of a term
    assert np.all(np.abs(_np(f["weights"]) - want["weights"]) <= 64 * U * want["weights"] + 1e-37)
    dl = OM.route_backward(ln, want["experts"], _np(d), scoring, normalize)
    mag = np.abs(_np(d)).max(1)[:, None] * (np.abs(dl) > 0)
    assert np.all(np.abs(_np(got) - dl) <= 128 * U * mag + U * np.abs(dl) + 1e-37)
    assert (np.abs(dl[:, :2]).max() > 0) == (scoring == "softmax" and not normalize)
    if not normalize:                                    # ... which is the difference quotient's answer too
        h, t = 1e-6, 7
        for e in (0, 1, int(want["experts"][t, 0])):
            up, dn = ln[t].astype(np.float64), ln[t].astype(np.float64)
            up[e] += h
            dn[e] -= h
            p = [OM.probabilities(v, want["experts"][t], scoring, normalize)[want["experts"][t]] for v in (up, dn)]
            assert abs(((p[0] - p[1]) * _np(d)[t]).sum() / (2 * h) - dl[t, e]) < 1e-7
