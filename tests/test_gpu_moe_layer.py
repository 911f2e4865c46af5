"""The expert MLP block end to end: each product recomputed in float64 from the
layer's own quantized operands, the routing against the oracle, a closed-form
check of the whole at high precision weights, and repeatability."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from fp8_quantized_gemm_amd.moe import MoELayer
from oracle import gemm as OG
from oracle import mlp as OMLP
from oracle import moe as OM
from oracle import norm as ON

from _gpu import announce, bits, gpu

pytestmark = gpu


def _np(t):
    return t.detach().double().cpu().numpy()


def _layer(E=6, F=96, Hd=160, k=2, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    norm = dict(w_pre=1 + 0.1 * rn(Hd), w_post=1 + 0.1 * rn(Hd), gate=rn(Hd), alpha=0.9, eps=1e-5)
    return MoELayer(0.05 * rn(E, 2 * F, Hd), 0.05 * rn(E, Hd, F), k, norm, rht_signs=0x5A3C, sr_seed=11, **kw), rn


def _deq(q, side):
    return OG.dequant_nvfp4(q[side + "_codes"].cpu().numpy(), q[side + "_scales"].cpu().numpy())


def _deq_w(w, side):
    c, s = w[side + "c"].cpu().numpy(), w[side + "s"].cpu().numpy()
    return np.stack([OG.dequant_nvfp4(c[e], s[e]) for e in range(len(c))])


@pytest.mark.parametrize("T,k,scoring", [(1, 2, "softmax"), (75, 2, "softmax"), (300, 3, "sigmoid")])
def test_step(T, k, scoring):
    announce("MoELayer step", T, k, scoring)
    L, rn = _layer(k=k, scoring=scoring)
    x, o, d_y = rn(T, L.Hd).bfloat16(), rn(T, L.Hd).bfloat16(), rn(T, L.Hd).bfloat16()
    logits = 2 * rn(T, L.E)
    if T > 2:
        logits[1] = float("-inf")                        # a token without experts
    r, h = L.open(x, o)
    y = L.forward(h, logits)
    d_h, d_logits = L.backward(d_y)
    grads = L.close(d_y, d_h)
    torch.cuda.synchronize()

    off = L.route["offsets"].cpu().numpy()
    w = OM.route(logits.cpu().numpy(), k, None, scoring, True, 1.0, 32)
    assert np.array_equal(L.route["src"].cpu().numpy(), w["src"]) and np.array_equal(off, w["offsets"])
    alpha = lambda a, b: OG.nvfp4_alpha(np.float32(a.item()), np.float32(b.item()))

    def rows(q, n, side, got, what):
        want, _ = OM.grouped(_deq(q, "row"), _deq_w(L.wq[n], side), off)
        rep = OG.tolerance_report(_np(got), want * alpha(q["row_amax"], L.wamax[n]))
        assert rep["passed"], (what, rep)
    rows(L.qx, "W_gu", "r", L.y_gu, "Y_gu")
    rows(L.qh, "W_down", "r", L.y_down, "Y_down")

    def cols(qa, qb, n):
        want, _ = OM.grouped_wgrad(_deq(qa, "col"), _deq(qb, "col"), off)
        rep = OG.tolerance_report(_np(L.grad[n]), want * alpha(qa["col_amax"], qb["col_amax"]))
        assert rep["passed"], (n, rep)
    cols(L.qd, L.qh, "W_down")
    cols(L.qg, L.qx, "W_gu")

    # combine with the routing weights, from the layer's own Y_down
    want = OM.combine(_np(L.y_down), L.route["row_of"].cpu().numpy(), _np(L.route["weights"]))
    assert np.all(np.abs(_np(y) - want) <= 2.0 ** -7 * np.abs(want) + 1e-6)
    if T > 2:
        assert not y[1].any() and not d_h[1].any() and not d_logits[1].any()
    # the norm around it
    f = ON.forward(_np(x), _np(o), _np(L.norm["w_pre"]), _np(L.norm["w_post"]), _np(L.norm["gate"]), 0.9, 1e-5)
    assert np.allclose(_np(h), f["h"], rtol=2.0 ** -7, atol=1e-4) and np.allclose(_np(r), f["r"], rtol=2.0 ** -7, atol=1e-4)
    assert all(torch.isfinite(v).all() for v in grads.values() if v is not None)


def test_matches_the_unquantized_block():
    """Against the float64 block on the unquantized weights: each of the two products
    carries the relative error of two NVFP4 operands (element steps of 1/4 to 1/8,
    0.1 rms each), so y is within 0.3 relative of the exact one in the 2-norm."""
    announce("MoELayer against the unquantized block")
    L, rn = _layer(E=4, F=128, Hd=256, k=2, seed=3, normalize=True)
    h, logits = rn(200, 256).bfloat16(), rn(200, 4)
    y = _np(L.forward(h, logits))
    wg, wd = _np(L.wbf["W_gu"]), _np(L.wbf["W_down"])
    r = OM.route(logits.cpu().numpy(), 2)
    want = np.zeros_like(y)
    for t in range(200):
        for j in range(2):
            z = wg[r["experts"][t, j]] @ _np(h)[t]
            a = OMLP.silu_f64(z[:128]) * z[128:]
            want[t] += r["weights"][t, j] * (wd[r["experts"][t, j]] @ a)
    assert np.linalg.norm(y - want) < 0.3 * np.linalg.norm(want)


def test_same_bits_and_update():
    announce("MoELayer repeats and updates")
    out = []
    for _ in range(2):
        L, rn = _layer(seed=7)
        x, o = rn(90, L.Hd).bfloat16(), rn(90, L.Hd).bfloat16()
        logits, d_y = rn(90, L.E), rn(90, L.Hd).bfloat16()
        vals = []
        for _ in range(2):
            _, h = L.open(x, o)
            y = L.forward(h, logits)
            d_h, d_l = L.backward(d_y)
            L.close(d_y, d_h)
            w = L.w32["W_gu"].clone()
            L.update()
            assert not torch.equal(w, L.w32["W_gu"])
            assert np.array_equal(bits(L.wbf["W_gu"]), bits(L.w32["W_gu"].bfloat16()))
            vals += [y, d_h, d_l, L.grad["W_gu"].clone(), L.grad["W_down"].clone()]
        out.append(vals)
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_refusals():
    w = torch.zeros((2, 64, 32), device="cuda")
    with pytest.raises(ValueError):
        MoELayer(w, torch.zeros((2, 32, 16), device="cuda"), 1, dict(w_pre=torch.ones(32, device="cuda")))
    with pytest.raises(ValueError):
        MoELayer(w, torch.zeros((2, 32, 32), device="cuda"), 1, dict())
    with pytest.raises(bsq.BsqError):
        MoELayer(w, torch.zeros((2, 32, 32), device="cuda"), 3, dict(w_pre=torch.ones(32, device="cuda"))).forward(
            torch.zeros((4, 32), device="cuda").bfloat16(), torch.zeros((4, 2), device="cuda"))
