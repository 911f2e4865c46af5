"""The 8-bit products and the orthogonalised update in use: training steps of the MLP and
of the expert block that run on them.

Each link is held against the oracle on the layer's own tensors: the quantizers and the
products bit for bit, SwiGLU to one step of BF16 (what swiglu_amax promises), the momentum
bit for bit, the weights to the tolerance of test_gpu_muon (twice the distance that the
FP16 roundings alone cause, plus FP16's half step and the FP32 roundings)."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from fp8_quantized_gemm_amd.mlp import MLPLayer
from fp8_quantized_gemm_amd.moe import MoELayer
from oracle import int8 as O8
from oracle import mlp as M
from oracle import muon as OM

from _gpu import announce, assert_bytes_equal, bits, gpu

pytestmark = gpu


def _np(t):
    return t.detach().float().cpu().numpy()


def _mlp(T, Hd, F, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)
    L = MLPLayer((0.05 * rn(2 * F, Hd)).cuda(), (0.05 * rn(Hd, F)).cuda(), T, **kw)
    return L, lambda: (rn(T, Hd).bfloat16().cuda(), (1e-2 * rn(T, Hd)).bfloat16().cuda())


def _operand(L, name, x):
    """The layer's codes and scales of both sides, after a check against the oracle."""
    q, b = L.q[name], bits(x)
    for side, v in (("r", b), ("c", np.ascontiguousarray(b.T))):
        codes, scales = O8.quantize(v)
        assert np.array_equal(q[side + "c"].cpu().numpy(), codes), (name, side)
        assert np.array_equal(q[side + "s"].cpu().numpy(), scales), (name, side)
    return {s: (q[s + "c"].cpu().numpy(), q[s + "s"].cpu().numpy()) for s in "rc"}


def _product(got, a, b, what):
    assert np.array_equal(_np(got), O8.gemm(*a, *b).astype(np.float32)), what


def _one_step(got, want, what):
    """BF16 bit patterns at most one value apart (two zeros count as one)."""
    order = lambda v: np.where(v & 0x8000, -(v & 0x7FFF).astype(np.int32), (v & 0x7FFF).astype(np.int32))
    assert np.abs(order(got) - order(want)).max() <= 1, what


def _check_muon(before, after, grad, lr, o, what):
    """One update of a stack [B, R, C]: (w, momentum) before and after."""
    (w, m), (wn, mn) = before, after
    f = np.float32
    em, u = OM.moment(m, grad, o["mu"], o["nesterov"])
    assert np.array_equal(mn, em), what
    R, C = w.shape[-2:]
    step = float(f(f(lr) * f(0.2 * max(R, C) ** 0.5)))
    keep = float(f(1) - f(lr) * f(o["weight_decay"]))
    for wi, ui, yi in zip(w.astype(np.float64), u.astype(np.float64), wn.astype(np.float64)):
        e, n = OM.orthogonalize(ui), np.linalg.norm
        q = OM.orthogonalize_f16(ui, plan=OM.plan(R, C))
        tol = step * (2 * n(q - e) + 2.0 ** -11 * n(e)) + 2.0 ** -23 * (n(wi) + step * n(e))
        assert n(yi - (keep * wi - step * e)) <= tol, (what, n(yi - (keep * wi - step * e)), tol)


@pytest.mark.parametrize("T,Hd,F", [(16, 64, 32), (144, 160, 112), (272, 320, 208)])
def test_mlp_step(T, Hd, F):
    announce("MLPLayer int8 muon", T, Hd, F)
    o = dict(mu=0.9, nesterov=True, weight_decay=0.1)
    L, data = _mlp(T, Hd, F, fmt="int8", optimizer="muon", muon=o, lr=0.02)
    stacks = {"W_gu": (2, F, Hd), "W_down": (1, Hd, F)}
    for step in range(3):
        x, dy = data()
        used = {k: v.clone() for k, v in L.wbf.items()}
        before = {k: (_np(L.w32[k]).reshape(s), _np(L.momentum[k]).reshape(s)) for k, s in stacks.items()}
        y, dx = L.step(x, dy)
        torch.cuda.synchronize()
        act = L.act
        qx, qh = _operand(L, "X", x), _operand(L, "H", act["H"])
        qg, qd = _operand(L, "W_gu", used["W_gu"]), _operand(L, "W_down", used["W_down"])
        qy, qz = _operand(L, "dY_down", dy), _operand(L, "dY_gu", act["dY_gu"])
        _product(act["Y_gu"], qx["r"], qg["r"], "Y_gu")
        _one_step(bits(act["H"]), M.swiglu(bits(act["Y_gu"])), "H")
        _product(y, qh["r"], qd["r"], "Y_down")
        _product(act["dH"], qy["r"], qd["c"], "dH")
        _product(L.grad["W_down"], qy["c"], qh["c"], "dW_down")
        _one_step(bits(act["dY_gu"]), M.swiglu_backward(bits(act["Y_gu"]), bits(act["dH"])), "dY_gu")
        _product(dx, qz["r"], qg["c"], "dX")
        _product(L.grad["W_gu"], qz["c"], qx["c"], "dW_gu")
        for k, s in stacks.items():
            after = (_np(L.w32[k]).reshape(s), _np(L.momentum[k]).reshape(s))
            _check_muon(before[k], after, _np(L.grad[k]).reshape(s), 0.02, o, (k, step))
            assert torch.equal(L.wbf[k], L.w32[k].bfloat16())
            assert float(L.wamax[k]) == float(L.wbf[k].float().abs().max())


@pytest.mark.parametrize("fmt,optimizer", [("int8", "sgd"), ("nvfp4", "muon")])
def test_mlp_mixed(fmt, optimizer):
    """Either one alone: the other half is what it is without."""
    announce("MLPLayer", fmt, optimizer)
    L, data = _mlp(48, 64, 80, seed=3, fmt=fmt, optimizer=optimizer, lr=1e-2)
    P, _ = _mlp(48, 64, 80, seed=3, fmt=fmt, lr=1e-2) if fmt == "int8" else _mlp(48, 64, 80, seed=3, lr=1e-2)
    x, dy = data()
    for a, b in zip(L.step(x, dy), P.step(x, dy)):
        assert torch.equal(a, b)
    for k in L.w32:
        assert torch.equal(L.grad[k], P.grad[k])
        if optimizer == "sgd":
            assert torch.equal(L.w32[k], P.w32[k])
    if optimizer == "muon":
        s = {"W_gu": (2, 80, 64), "W_down": (1, 64, 80)}
        Q, _ = _mlp(48, 64, 80, seed=3)
        for k in L.w32:
            w, m = Q.w32[k].view(s[k]), torch.zeros_like(Q.w32[k]).view(s[k])
            bsq.muon_update(w, m, L.grad[k].view(s[k]), 1e-2)
            assert torch.equal(L.w32[k], Q.w32[k]) and torch.equal(L.momentum[k].view(s[k]), m)


def test_mlp_follows_the_exact_layer():
    """Against the FP64 layer on the same weights.  A code is off by at most half a step,
    amax / 254; with normal entries and 256 of them amax is about 3 sigma, so an operand's
    error is uniform of root mean square 3 sigma / 127 / sqrt(12) = 0.7% of its own, and amax
    stays below 6 sigma (1.4%).  Y_down passes through X, W_gu, H (a product of two normals:
    amax at most 36 of its sigma, 8.2%) and W_down: at most sqrt(2 * 1.4%^2 * 2 + 8.2%^2 +
    1.4%^2) with SwiGLU's gain of at most 2 on Y_gu's error, below 10%."""
    announce("MLPLayer int8 against FP64")
    L, data = _mlp(256, 256, 256, seed=5, fmt="int8")
    x, _ = data()
    y = _np(L.forward(x)).astype(np.float64)
    z = _np(x).astype(np.float64) @ _np(L.wbf["W_gu"]).astype(np.float64).T
    h = M.silu_f64(z[:, :256]) * z[:, 256:]
    want = h @ _np(L.wbf["W_down"]).astype(np.float64).T
    assert np.linalg.norm(y - want) <= 0.1 * np.linalg.norm(want)


def test_mlp_serves_single_tokens():
    """int8_linear with the weights that the layer quantized gives its rows."""
    announce("MLPLayer int8, int8_linear")
    L, data = _mlp(32, 128, 96, seed=6, fmt="int8")
    x, _ = data()
    L.forward(x)
    q = L.q["W_gu"]
    for rows in (slice(0, 1), slice(3, 20), slice(0, 32)):
        got = bsq.int8_linear(x[rows], q["rc"], q["rs"])
        assert torch.equal(got, L.act["Y_gu"][rows])
    q = L.q["W_down"]
    assert torch.equal(bsq.int8_linear(L.act["H"][:1], q["rc"], q["rs"]), L.act["Y_down"][:1])


def test_mlp_captured():
    """A captured step replayed among eager ones of a second layer."""
    announce("MLPLayer int8 muon captured")
    a, data = _mlp(64, 96, 160, seed=7, fmt="int8", optimizer="muon", lr=0.02)
    b, _ = _mlp(64, 96, 160, seed=7, fmt="int8", optimizer="muon", lr=0.02)
    x, dy = data()
    a.step(x, dy), b.step(x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(x, dy)
    for _ in range(4):
        u, v = data()
        x.copy_(u), dy.copy_(v)
        graph.replay()
        y, dx = b.step(u, v)
        torch.cuda.synchronize()
        assert torch.equal(a.act["Y_down"], y) and torch.equal(a.act["dX"], dx)
        for k in a.w32:
            assert torch.equal(a.w32[k], b.w32[k]) and torch.equal(a.momentum[k], b.momentum[k])
            assert torch.equal(a.wbf[k], b.wbf[k]) and torch.equal(a.wamax[k], b.wamax[k])


def test_moe_muon():
    announce("MoELayer muon")
    E, F, Hd = 5, 48, 96
    o = dict(mu=0.9, nesterov=False, weight_decay=0.05)
    g = torch.Generator(device="cuda").manual_seed(9)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = 0.05 * rn(E, 2 * F, Hd), 0.05 * rn(E, Hd, F)
    norm = dict(w_pre=torch.ones(Hd, device="cuda"))
    L = MoELayer(*w, 2, norm, optimizer="muon", muon=o, lr=0.02)
    P = MoELayer(*w, 2, norm, lr=0.02)
    stacks = {"W_gu": (2 * E, F, Hd), "W_down": (E, Hd, F)}
    for step in range(2):
        h, logits, dy = rn(60, Hd).bfloat16(), rn(60, E), 1e-2 * rn(60, Hd)
        logits[:, 3] = -1e9                                  # an expert without tokens: gradients of zero
        outs = [(l.forward(h, logits), *l.backward(dy.bfloat16())) for l in (L, P)]
        if step == 0:
            assert all(torch.equal(a, b) for a, b in zip(*outs))
        before = {k: (_np(L.w32[k]).reshape(s), _np(L.momentum[k]).reshape(s)) for k, s in stacks.items()}
        L.update(), P.update()
        for k, s in stacks.items():
            after = (_np(L.w32[k]).reshape(s), _np(L.momentum[k]).reshape(s))
            _check_muon(before[k], after, _np(L.grad[k]).reshape(s), 0.02, o, (k, step))
            assert_bytes_equal(bits(L.wbf[k]), bits(L.w32[k].bfloat16()), k)
            assert float(L.wamax[k]) == float(L.wbf[k].float().abs().max())


def test_refusals():
    w = torch.zeros((64, 32), device="cuda"), torch.zeros((32, 32), device="cuda")
    e = torch.zeros((2, 64, 32), device="cuda"), torch.zeros((2, 32, 32), device="cuda")
    norm = dict(w_pre=torch.ones(32, device="cuda"))
    for kw in (dict(fmt="int4"), dict(optimizer="adam"), dict(muon=dict(mu=0.9)),
               dict(optimizer="muon", muon=dict(beta=0.9)), dict(optimizer="muon", muon=dict(steps=0)),
               dict(optimizer="muon", muon=dict(coefs=(1.0, 2.0)))):
        with pytest.raises(ValueError):
            MLPLayer(*w, 16, **kw)
    with pytest.raises(ValueError):
        MLPLayer(*w, 24, fmt="int8")
    with pytest.raises(ValueError):
        MLPLayer(*w, 1 << 17, fmt="int8")
    for kw in (dict(optimizer="adam"), dict(muon={}), dict(optimizer="muon", muon=dict(lr=1.0)),
               dict(optimizer="muon", muon=dict(steps=0))):
        with pytest.raises(ValueError):
            MoELayer(*e, 1, norm, **kw)
