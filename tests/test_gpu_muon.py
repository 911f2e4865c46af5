"""Orthogonalisation and the weight update against the FP64 definition.

Tolerance of an orthogonalised matrix: the products take FP16 values (each rounding at
most 2^-11) between which parts are held more exactly.  The oracle repeats those roundings with FP64 sums; its
distance from the definition is the error they cause, on this matrix and with these
coefficients.  The kernels' sums are FP32, so their roundings fall elsewhere but are of
the same number and size: twice that distance is allowed, and half a step of the output
type (2^-8 BF16, 2^-11 for the FP16 form of an update) of its norm."""

import math

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from _gpu import announce, gpu
from oracle import muon as OM

pytestmark = gpu


def _grad(shape, seed, dtype=torch.float32, size=1e-3):
    """A few strong directions over a broad floor, for each matrix of the stack."""
    g = torch.Generator().manual_seed(seed)
    *e, r, c = shape
    k = max(1, min(r, c) // 16)
    x = torch.randn((*e, r, k), generator=g) @ torch.randn((*e, k, c), generator=g) * (2 / math.sqrt(k))
    return ((x + torch.randn(shape, generator=g)) * size).to(dtype)


def _allowed(x, e, steps, coefs, eps, half_step, plan=None):
    f = OM.orthogonalize_f16(x, steps, coefs, eps, plan=plan or OM.plan(*x.shape, steps, coefs))
    n = np.linalg.norm(e)
    return 2 * np.linalg.norm(f - e) + half_step * n + 1e-30


def _check(x, steps=5, coefs=OM.COEFS, eps=1e-7):
    announce("orthogonalize", tuple(x.shape), x.dtype, steps)
    got = bsq.orthogonalize(x.cuda(), steps=steps, coefs=coefs, eps=eps)
    assert got.dtype == torch.bfloat16 and got.shape == x.shape
    xs, gs = x.double().numpy(), got.double().cpu().numpy()
    if x.dim() == 2:
        xs, gs = xs[None], gs[None]
    for m, y in zip(xs, gs):
        e = OM.orthogonalize(m, steps, coefs, eps)
        err, tol = np.linalg.norm(y - e), _allowed(m, e, steps, coefs, eps, 2.0 ** -8)
        assert err <= tol, (x.shape, err / np.linalg.norm(e), tol / np.linalg.norm(e))
    return got


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (2, 3), (16, 16), (63, 64), (64, 65), (65, 64), (64, 128), (128, 64),
                                   (100, 37), (37, 100), (200, 136), (129, 385), (256, 256), (257, 300), (520, 1000), (700, 200),
                                   (3, 1000), (1000, 5), (512, 640),
                                   # at and past the edges of what one workgroup holds
                                   (160, 160), (161, 161), (192, 200), (160, 256), (256, 161), (257, 150), (96, 512), (97, 512), (513, 90),
                                   (32, 1024), (1024, 33), (17, 1024), (1025, 16), (81, 449), (64, 768), (769, 64),
                                   (128, 250), (250, 129)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize(shape, dtype):
    _check(_grad(shape, 1, dtype))


@pytest.mark.parametrize("shape", [(1, 64, 64), (3, 65, 130), (5, 96, 32), (17, 24, 40), (2, 300, 260)])
def test_stacks(shape):
    x = _grad(shape, 2)
    got = _check(x)
    for i in range(shape[0]):                                # each matrix as if it were alone
        assert torch.equal(got[i], bsq.orthogonalize(x[i].cuda()))


@pytest.mark.parametrize("shape", [(96, 96), (64, 256), (256, 64), (300, 500), (448, 310)])
@pytest.mark.parametrize("steps,coefs", [
    (1, OM.COEFS), (2, OM.COEFS), (3, OM.COEFS), (8, OM.COEFS), (12, (1.5, -0.5, 0.0)), (6, (2.0, -1.5, 0.5)),
    (4, ((8.2, -23.0, 16.7), (4.1, -2.9, 0.53), (3.9, -2.8, 0.53), (1.9, -1.3, 0.4)))])
def test_steps_and_coefficients(shape, steps, coefs):
    _check(_grad(shape, 3), steps=steps, coefs=coefs)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e15, 1e30])
def test_sizes_of_values(size):
    """The norm is a sum of 64 bits: neither tiny nor huge matrices lose it."""
    _check(_grad((70, 90), 4, size=size), eps=1e-37)


def test_largest_epsilon():
    _check(_grad((70, 90), 5), eps=1.0)                      # the norm is of the order of eps


def test_known_matrices():
    """Matrices whose singular values are all equal, 1 / sqrt(n): the step's polynomial is
    one number, and FP16 holds every entry between products to 2^-11."""
    s = 1 / 8.0
    for a, b, c in (OM.COEFS,) * 5:
        s = a * s + b * s ** 3 + c * s ** 5
    perm = torch.randperm(64, generator=torch.Generator().manual_seed(6))
    p = torch.eye(64)[perm] * 3.0
    got = bsq.orthogonalize(p.cuda()).double().cpu()
    assert torch.equal(got != 0, p != 0)
    # |p'| <= 3.45 per step: each rounding grows at most so, 4 roundings a step
    tol = sum(4 * 2.0 ** -11 * 3.45 ** k for k in range(5)) + 2.0 ** -8
    assert float((got[p != 0] / s - 1).abs().max()) <= tol


def test_zero_and_non_finite():
    x = _grad((4, 66, 80), 7)
    x[1] = 0
    clean = bsq.orthogonalize(x.cuda())
    assert bool((clean[1] == 0).all())
    x[2, 5, 5] = float("nan")
    x[3, 0, 0] = float("inf")
    got = bsq.orthogonalize(x.cuda())
    assert torch.equal(got[0], clean[0]) and bool((got[1] == 0).all())
    assert bool(got[2].isnan().any()) and bool(got[3].isnan().any())


def test_empty():
    for shape in ((0, 5), (5, 0), (0, 4, 4), (2, 0, 4)):
        assert bsq.orthogonalize(torch.empty(shape, device="cuda")).shape == shape


def test_out_and_strides():
    x = _grad((90, 120), 8).cuda()
    want = bsq.orthogonalize(x)
    out = torch.empty(90, 120, dtype=torch.bfloat16, device="cuda")
    assert bsq.orthogonalize(x, out=out).data_ptr() == out.data_ptr() and torch.equal(out, want)
    assert torch.equal(bsq.orthogonalize(x.t().contiguous().t()), want)          # another memory order
    odd = torch.empty(90 * 120 + 1, device="cuda")[1:].view(90, 120)              # 4-byte alignment only
    odd.copy_(x)
    assert torch.equal(bsq.orthogonalize(odd), want)
    with pytest.raises(ValueError):
        bsq.orthogonalize(x, out=out.t())
    with pytest.raises(ValueError):
        bsq.orthogonalize(x.half())
    with pytest.raises(ValueError):
        bsq.orthogonalize(x, coefs=(1.0, 2.0))
    with pytest.raises(bsq.BsqError):
        bsq.orthogonalize(x, eps=0.0)


def _update_case(shape, seed):
    w = 0.02 * torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    return w, _grad(shape, seed + 1) * 5, _grad(shape, seed + 2, torch.bfloat16)


def _check_update(w, m, g, lr=1e-2, mu=0.95, nesterov=True, wd=0.1, scale=None):
    announce("muon_update", tuple(w.shape), nesterov)
    wd_, md = w.cuda(), m.cuda()
    got = bsq.muon_update(wd_, md, g.cuda(), lr, mu=mu, nesterov=nesterov, weight_decay=wd, scale=scale)
    f = np.float32
    em, u = OM.moment(m.numpy(), g.float().numpy(), mu, nesterov)
    assert np.array_equal(md.cpu().numpy(), em), "momentum"
    R, C = w.shape[-2:]
    step = float(f(f(lr) * f(0.2 * max(R, C) ** 0.5 if scale is None else scale)))
    keep = float(f(1) - f(lr) * f(wd))
    flat = lambda t: np.asarray(t, dtype=np.float64).reshape(-1, R, C)
    for wi, ui, yi in zip(flat(w), flat(u), flat(wd_.cpu())):
        e = OM.orthogonalize(ui)
        want = keep * wi - step * e
        # two products and a difference in FP32: 2^-24 of each
        tol = step * _allowed(ui, e, 5, OM.COEFS, 1e-7, 2.0 ** -11) + 2.0 ** -23 * (np.linalg.norm(wi) + step * np.linalg.norm(e))
        assert np.linalg.norm(yi - want) <= tol, (w.shape, np.linalg.norm(yi - want), tol)
    assert torch.equal(got["w_bf16"], wd_.bfloat16())
    assert float(got["amax"]) == float(got["w_bf16"].float().abs().max())
    return wd_, md


@pytest.mark.parametrize("shape", [(1, 1), (7, 5), (64, 64), (65, 129), (200, 136), (136, 200), (512, 256), (256, 700),
                                   (3, 66, 100), (2, 520, 1000), (9, 40, 24)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_update(shape, nesterov):
    _check_update(*_update_case(shape, 20), nesterov=nesterov)


def test_update_arguments():
    w, m, g = _update_case((96, 160), 30)
    _check_update(w, m, g, mu=0.0, wd=0.0, scale=1.0)
    w0, m0 = w.cuda(), m.cuda()
    u = bsq.muon_update(w0, m0, g.cuda(), 0.0, amax=False)   # lr 0: the weight stays, the momentum moves
    assert torch.equal(w0.cpu(), w) and u["amax"] is None and not torch.equal(m0.cpu(), m)
    zero = torch.zeros_like(w).cuda()
    bsq.muon_update(w0, zero.clone(), zero.bfloat16(), 1e-2)  # nothing to follow
    assert torch.equal(w0.cpu(), w)
    wb = torch.empty(96, 160, dtype=torch.bfloat16, device="cuda")
    assert bsq.muon_update(w0, m0, g.cuda(), 1e-2, w_bf16=wb)["w_bf16"].data_ptr() == wb.data_ptr()
    with pytest.raises(ValueError):
        bsq.muon_update(w0.t(), m0, g.cuda(), 1e-2)
    with pytest.raises(ValueError):
        bsq.muon_update(w0, m0[:90], g.cuda(), 1e-2)
    with pytest.raises(ValueError):
        bsq.muon_update(w0, m0, g.float().cuda(), 1e-2)
    with pytest.raises(bsq.BsqError):
        bsq.muon_update(w0, w0, g.cuda(), 1e-2)              # one tensor twice


def test_update_repeats_bit_for_bit():
    w, m, g = _update_case((2, 300, 200), 40)
    a = _check_update(w, m, g)
    for _ in range(3):
        wd, md = w.cuda(), m.cuda()
        bsq.muon_update(wd, md, g.cuda(), 1e-2, weight_decay=0.1)
        assert torch.equal(wd, a[0]) and torch.equal(md, a[1])


def test_streams_and_graph():
    x = _grad((150, 260), 50).cuda()
    want = bsq.orthogonalize(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = bsq.orthogonalize(x)
    s.synchronize()
    assert torch.equal(y, want)
    w, m, g = (t.cuda() for t in _update_case((150, 260), 51))
    we, me = w.clone(), m.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = bsq.orthogonalize(x)
        u = bsq.muon_update(w, m, g, 1e-2)
    for i in range(4):
        x.copy_(_grad((150, 260), 60 + i))
        g.copy_(_grad((150, 260), 70 + i, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bsq.orthogonalize(x))
        e = bsq.muon_update(we, me, g, 1e-2)
        assert torch.equal(w, we) and torch.equal(m, me)
        assert torch.equal(u["w_bf16"], e["w_bf16"]) and torch.equal(u["amax"], e["amax"])


@pytest.mark.parametrize("shape", [(120, 200), (3, 64, 90), (330, 500)])
def test_two_at_once_and_captured(shape):
    """Both forms (one workgroup, many launches): updates of two weights on two streams at
    the same time, and replays of a captured one, against the same calls one by one."""
    announce("muon_update, two at once", shape)
    cases = [[t.cuda() for t in _update_case(shape, 80 + i)] for i in range(2)]
    want = [[t.clone() for t in c] for c in cases]
    for w, m, g in want:
        for _ in range(3):
            bsq.muon_update(w, m, g, 1e-2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for _ in range(3):
        for s, (w, m, g) in zip(streams, cases):
            with torch.cuda.stream(s):
                outs.append(bsq.muon_update(w, m, g, 1e-2))
    torch.cuda.synchronize()
    for (w, m, _), (we, me, _) in zip(cases, want):
        assert torch.equal(w, we) and torch.equal(m, me)
    for u, (w, _, _) in zip(outs[-2:], cases):
        assert torch.equal(u["w_bf16"], w.bfloat16()) and float(u["amax"]) == float(u["w_bf16"].float().abs().max())
    (w, m, g), (we, me, _) = cases[0], want[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        u = bsq.muon_update(w, m, g, 1e-2)
    for i in range(4):
        g.copy_(_grad(shape, 90 + i, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        e = bsq.muon_update(we, me, g, 1e-2)
        assert torch.equal(w, we) and torch.equal(m, me)
        assert torch.equal(u["w_bf16"], e["w_bf16"]) and torch.equal(u["amax"], e["amax"])


def test_one_workgroup_form_unaligned():
    """Updates at addresses that only their type aligns, and the refusal of a result over its input."""
    w, m, g = _update_case((75, 130), 95)
    want = _check_update(w, m, g)
    odd = lambda t: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    wo, mo, wb = odd(w), odd(m), odd(g)
    u = bsq.muon_update(wo, mo, odd(g), 1e-2, weight_decay=0.1, w_bf16=wb)
    assert torch.equal(wo, want[0]) and torch.equal(mo, want[1]) and torch.equal(u["w_bf16"], wo.bfloat16())
    x = _grad((75, 130), 96, torch.bfloat16).cuda()
    x0 = x.clone()
    with pytest.raises(bsq.BsqError):
        bsq.orthogonalize(x, out=x)
    torch.cuda.synchronize()
    assert torch.equal(x, x0)
