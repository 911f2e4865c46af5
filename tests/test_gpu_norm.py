"""block_norm and its gradient against the float64 oracle.

Tolerances: every FP32 operation is off by at most 2^-24 relative; a row mean is a
tree of at most 16 serial and 6 + 16 joining additions, so 64 such steps cover a
value's arithmetic, relative to the sum of the absolute values of its terms.
Column sums add at most rows / 512 + 32 partials: 192 steps.  A BF16 output adds
half a step, 2^-8 relative."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from oracle import norm as ON

from _gpu import announce, gpu

pytestmark = gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _inputs(R, C, res, gate, post, pre, has_o, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    t = TYPES[res]
    i = dict(x=(rn(R, C) * 2).to(t), o=(rn(R, C) * 3).bfloat16() if has_o else None,
             w_pre=1 + 0.3 * rn(C) if pre else None, w_post=1 + 0.3 * rn(C) if post else None, gate=None)
    if gate == "channel":
        i["gate"] = rn(C)
    elif gate == "row":
        i["gate"] = rn(R, 1)
    elif gate == "full":
        i["gate"] = rn(R, C).bfloat16()
    i["d_r"] = rn(R, C).to(t)
    i["d_h"] = rn(R, C).bfloat16() if pre else None
    return i


def _close(got, want, mag, steps, what):
    got = _np(got)
    half = 2.0 ** -8 if what.endswith("bf16") else U
    # the stored value's own rounding is relative to the value before it
    tol = steps * U * mag + half * (np.abs(want) + steps * U * mag) + 1e-40
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - want) - tol)))


CASES = [  # rows, cols, residual, gate, post, pre, o
    (1, 1, "f32", None, True, True, True),
    (1, 4096, "bf16", None, True, True, True),
    (3, 8, "bf16", "channel", True, True, True),
    (5, 97, "f32", "row", True, True, True),
    (130, 512, "bf16", "full", True, True, True),
    (67, 520, "f32", "channel", False, True, True),
    (33, 1000, "bf16", "row", False, True, True),
    (1100, 2048, "f32", "full", True, True, True),
    (9, 2049, "bf16", "channel", True, True, True),
    (600, 4096, "bf16", "channel", True, False, True),
    (17, 5000, "f32", None, True, True, True),
    (3, 8191, "bf16", "channel", True, True, True),
    (4, 16384, "f32", "channel", True, True, True),
    (2, 16383, "bf16", "full", True, True, True),
    (515, 1408, "bf16", None, False, True, False),
    (70, 64, "f32", None, False, True, False),
    (2, 63, "bf16", None, False, False, True),
    (1000, 127, "bf16", "channel", True, True, True),
    (301, 128, "f32", "row", True, True, True),
    (77, 200, "bf16", "full", True, True, True),
    (50, 256, "f32", None, True, True, True),
    (40, 1024, "bf16", "channel", True, True, True),
    (21, 8192, "f32", "full", True, True, True),
    (19, 12000, "bf16", "row", True, True, True),
    (600, 9000, "f32", "channel", True, True, True),
    (530, 16384, "bf16", "full", True, True, True),
    (300, 8203, "bf16", None, False, True, True),
]


@pytest.mark.parametrize("R,C,res,gate,post,pre,has_o", CASES)
def test_forward(R, C, res, gate, post, pre, has_o):
    announce("block_norm", R, C, res, gate, post, pre, has_o)
    i = _inputs(R, C, res, gate, post, pre, has_o, 11 + C)
    f = bsq.block_norm(i["x"], i["o"], i["w_pre"], i["w_post"], i["gate"], alpha=0.75, eps=1e-5, amax=True)
    x, o, wp, wq, g = (_np(i[k]) for k in ("x", "o", "w_pre", "w_post", "gate"))
    w = ON.forward(x, o, wp, wq, g, alpha=np.float64(0.75), eps=float(np.float32(1e-5)))
    assert (f["r"] is None) == (w["r"] is None) and (f["h"] is None) == (w["h"] is None)
    mag = np.abs(x)
    if has_o:
        n = o if wq is None else o * w["rstd_post"][:, None] * wq
        mag = 0.75 * np.abs(x) + np.abs(n if g is None else g * n)
        assert f["r"].dtype == i["x"].dtype
        _close(f["r"], w["r"], mag, 64, "r " + res)
    if post:
        _close(f["rstd_post"], w["rstd_post"], w["rstd_post"], 64, "rstd_post f32")
    if pre:
        # relative error of rstd: that of the mean of squares, |r| dr summed over r^2
        rel = (mag * np.abs(w["r"] if has_o else x)).sum(1) / np.maximum(((w["r"] if has_o else x) ** 2).sum(1), 1e-300)
        _close(f["rstd_pre"], w["rstd_pre"], w["rstd_pre"] * (1 + rel), 64, "rstd_pre f32")
        k = np.abs(w["rstd_pre"])[:, None] * np.abs(wp)
        _close(f["h"], w["h"], k * (mag + np.abs(w["r"] if has_o else x) * (1 + rel[:, None])), 64, "h bf16")
        assert f["amax"].item() == f["h"].abs().max().item()
    else:
        assert f["amax"] is None and f["rstd_pre"] is None


@pytest.mark.parametrize("R,C,res,gate,post,pre,has_o", CASES)
def test_backward(R, C, res, gate, post, pre, has_o):
    announce("block_norm_backward", R, C, res, gate, post, pre, has_o)
    i = _inputs(R, C, res, gate, post, pre, has_o, 12 + C)
    f = bsq.block_norm(i["x"], i["o"], i["w_pre"], i["w_post"], i["gate"], alpha=0.75)
    r = f["r"] if has_o else i["x"]
    kw = dict(o=i["o"], d_r=i["d_r"], d_h=i["d_h"], w_pre=i["w_pre"], w_post=i["w_post"], gate=i["gate"],
              rstd_pre=f["rstd_pre"], rstd_post=f["rstd_post"])
    b = bsq.block_norm_backward(r, alpha=0.75, **kw)
    want = ON.backward(_np(r), alpha=0.75, **{k: _np(v) for k, v in kw.items()})
    for name, t in b.items():
        if name not in want:
            assert t is None, name
            continue
        steps = 192 if name in ("d_w_pre", "d_w_post") or (name == "d_gate" and gate == "channel") else 64
        kind = "bf16" if t.dtype == torch.bfloat16 else "f32"
        # four values are summed for the two means of a row
        _close(t, want[name], want[name + "_"], 4 * steps, f"{name} {kind}")
    again = bsq.block_norm_backward(r, alpha=0.75, **kw)
    for name, t in b.items():
        assert t is None or torch.equal(t, again[name]), f"{name} differs from call to call"


def test_without_incoming_residual_gradient():
    announce("block_norm_backward, d_r absent")
    i = _inputs(37, 640, "bf16", "channel", True, True, True, 5)
    f = bsq.block_norm(i["x"], i["o"], i["w_pre"], i["w_post"], i["gate"])
    kw = dict(o=i["o"], d_h=i["d_h"], w_pre=i["w_pre"], w_post=i["w_post"], gate=i["gate"], rstd_pre=f["rstd_pre"],
              rstd_post=f["rstd_post"])
    none = bsq.block_norm_backward(f["r"], **kw)
    zero = bsq.block_norm_backward(f["r"], d_r=torch.zeros_like(f["r"]), **kw)
    for k in none:
        assert torch.equal(none[k], zero[k]), k


def test_gradient_is_the_difference_quotient():
    """FP32 residual, FP32 losses by differences of the library's own forward: with a
    step of 2^-6 on parameters of size 1 the quotient of the FP32 r is off by 2^-18
    relative at most; the BF16 h is left out of the loss."""
    announce("block_norm differences")
    g = torch.Generator(device="cuda").manual_seed(9)
    R, C = 6, 40
    x, o = torch.randn((R, C), generator=g, device="cuda"), torch.randn((R, C), generator=g, device="cuda").bfloat16()
    wq, gate = 1 + 0.2 * torch.randn(C, generator=g, device="cuda"), torch.randn(C, generator=g, device="cuda")
    d_r = torch.randn((R, C), generator=g, device="cuda")
    f = bsq.block_norm(x, o, w_post=wq, gate=gate, alpha=0.5)
    b = bsq.block_norm_backward(f["r"], o=o, d_r=d_r, w_post=wq, gate=gate, rstd_post=f["rstd_post"], alpha=0.5)
    h = 2.0 ** -6
    loss = lambda: (bsq.block_norm(x, o, w_post=wq, gate=gate, alpha=0.5)["r"].double() * d_r.double()).sum().item()
    for v, name in ((gate, "d_gate"), (wq, "d_w_post")):
        for c in (0, 17, 39):
            keep = v[c].item()
            v[c] = keep + h
            up = loss()
            v[c] = keep - h
            down = loss()
            v[c] = keep
            # r is linear in the gate and in w_post; loss error <= R * |d_r r| * 2^-23 / 2^-5
            assert abs((up - down) / (2 * h) - b[name][c].item()) < 2.0 ** -12, (name, c)


def test_zero_rows_and_extremes():
    announce("block_norm zero rows, zero row values, large values")
    w = torch.ones(64, device="cuda")
    f = bsq.block_norm(torch.zeros((0, 64), device="cuda"), torch.zeros((0, 64), device="cuda").bfloat16(), w, w, amax=True)
    assert f["r"].shape == (0, 64) and f["amax"].item() == 0
    b = bsq.block_norm_backward(f["r"], o=f["h"], d_r=f["r"], d_h=f["h"], w_pre=w, w_post=w, rstd_pre=f["rstd_pre"],
                                rstd_post=f["rstd_post"])
    assert not b["d_w_pre"].any() and not b["d_w_post"].any()
    x = torch.zeros((2, 64), device="cuda")
    x[1] = 1e15
    f = bsq.block_norm(x, w_pre=w)                       # a zero row stays zero, a large one has norm 1
    assert not f["h"][0].any() and torch.all(f["h"][1] == 1)


def test_unaligned_views_and_strides():
    announce("block_norm on views")
    base = torch.randn((10, 72), device="cuda").bfloat16()
    x = base[1:, 3:67]                                   # strided view: taken as a contiguous copy
    w = torch.randn(65, device="cuda")[1:]               # 4-byte aligned only
    a = bsq.block_norm(x, x, w, w)
    c = bsq.block_norm(x.contiguous(), x.contiguous(), w.clone(), w.clone())
    for k in ("r", "h"):                                 # another split of the sums: one BF16 step at most
        d = (a[k].float() - c[k].float()).abs()
        assert torch.all(d <= 2.0 ** -7 * c[k].float().abs() + 1e-30), k


def test_refusals():
    x = torch.zeros((4, 64), device="cuda").bfloat16()
    w = torch.ones(64, device="cuda")
    for kw in (dict(w_pre=w[:63]), dict(w_pre=w.bfloat16()), dict(w_pre=w, o=x[:3]), dict(w_pre=w, o=x, gate=w[:5]),
               dict(w_pre=w, o=x.float())):
        with pytest.raises(ValueError):
            bsq.block_norm(x, **kw)
    with pytest.raises(bsq.BsqError):
        bsq.block_norm(x)                                # nothing to compute
    with pytest.raises(ValueError):
        bsq.block_norm(x.half(), w_pre=w)


def test_other_stream_and_graph():
    announce("block_norm on another stream and in a graph")
    i = _inputs(48, 1024, "bf16", "channel", True, True, True, 8)
    call = lambda: bsq.block_norm(i["x"], i["o"], i["w_pre"], i["w_post"], i["gate"], amax=True)
    back = lambda f: bsq.block_norm_backward(f["r"], o=i["o"], d_r=i["d_r"], d_h=i["d_h"], w_pre=i["w_pre"],
                                             w_post=i["w_post"], gate=i["gate"], rstd_pre=f["rstd_pre"],
                                             rstd_post=f["rstd_post"])
    f = call()
    want = {**f, **back(f)}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f = call()
        got = {**f, **back(f)}
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = call()
        rec = {**f, **back(f)}
    for n in range(3):
        for t in rec.values():
            if t is not None:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            assert v is None or (torch.equal(v, got[k]) and torch.equal(v, rec[k])), (n, k)
        call()
