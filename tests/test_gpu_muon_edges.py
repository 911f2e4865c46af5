"""The orthogonalisation and its update where the values are extreme, in both forms: one
workgroup, single steps by products, and pairs of steps by products.  Tolerances are
those of test_gpu_muon."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from _gpu import announce, gpu
from test_gpu_muon import _check, _check_update, _grad, _update_case

pytestmark = gpu

# one workgroup; products, one step at a time; products, pairs of steps (and tall)
SHAPES = [(66, 80), (200, 330), (300, 500), (500, 300)]


@pytest.mark.parametrize("eps", [1e-37, 1.5e-45])
@pytest.mark.parametrize("shape", SHAPES)
def test_zero_and_tiny_matrices_under_a_tiny_epsilon(shape, eps):
    """1024 / (norm + eps) is above FP32 here: zeros stay zeros, and a matrix whose norm is
    of the order of 1e-37 (subnormal entries) is orthogonalised as any other."""
    announce("orthogonalize, tiny", shape, eps)
    zero = torch.zeros(shape, device="cuda")
    for x in (zero, zero.bfloat16()):
        assert bool((bsq.orthogonalize(x, eps=eps) == 0).all())
    x = _grad((2, *shape), 1, size=1e-39)
    assert 0 < float(x.double().norm()) < 3e-36
    x[1] = 0
    assert bool((_check(x, eps=eps)[1] == 0).all())


@pytest.mark.parametrize("shape", SHAPES)
def test_update_without_a_gradient_under_a_tiny_epsilon(shape):
    """Nothing to follow: the weights decay, and no more."""
    announce("muon_update, nothing to follow", shape)
    w = 0.02 * torch.randn(shape, generator=torch.Generator().manual_seed(2))
    wd, m, g = w.cuda(), torch.zeros(shape, device="cuda"), torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    u = bsq.muon_update(wd, m, g, 1e-2, weight_decay=0.1, eps=1e-37)
    keep = np.float32(1) - np.float32(1e-2) * np.float32(0.1)
    assert np.array_equal(wd.cpu().numpy(), keep * w.numpy()) and bool((m == 0).all())
    assert torch.equal(u["w_bf16"], wd.bfloat16()) and float(u["amax"]) == float(u["w_bf16"].float().abs().max())


@pytest.mark.parametrize("steps", [1, 4])
@pytest.mark.parametrize("shape", [*SHAPES, (320, 320), (640, 700)])
def test_entries_next_to_a_tie(shape, steps):
    """Steps that multiply X (a = 1.25, b = c = 0), read in FP32 from an update of zero
    weights: each entry is the scaled one to 22 bits (2^-22 a step, as much for the scaling
    and the norm), rounded to FP16 once (2^-11 of it, or 2^-25 below FP16's normal range, under
    the scale of 1,024).  An entry next to a tie of FP16 whose parts do not fit together is off
    by a whole FP16 step before that, 1.25 after."""
    announce("muon_update, steps that multiply", shape, steps)
    x = torch.randn(shape, generator=torch.Generator().manual_seed(3))
    w, m = torch.zeros(shape, device="cuda"), x.cuda()
    bsq.muon_update(w, m, torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), 1.0, mu=1.0, nesterov=False, scale=1.0,
                    steps=steps, coefs=(1.25, 0.0, 0.0))
    e = 1.25 ** steps * x.double() / (x.double().square().sum().sqrt() + float(np.float32(1e-7)))
    err = (-w.double().cpu() - e).abs() - (2.0 ** -11 + (steps + 2) * 2.0 ** -22) * e.abs() - 2.0 ** -35
    assert float(err.max()) <= 0, (shape, int((err > 0).sum()), float((err / e.abs()).max()))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["first", "last", "middle"])
@pytest.mark.parametrize("shape", [*SHAPES, (1, 2000), (1100, 1), (33, 1500), (700, 40)])
def test_non_finite_stays_in_its_matrix(shape, where, bad):
    """By the definition every entry of the matrix is NaN (its norm is NaN, or infinite, and
    the one entry that is then NaN reaches all others through A^2); the matrices beside it are
    what they are without it, bit for bit."""
    announce("orthogonalize, non-finite", shape, where, bad)
    R, C = shape
    r, c = dict(first=(0, 0), last=(R - 1, C - 1), middle=(R // 2, C // 2))[where]
    x = _grad((3, R, C), 4)
    x[2] = 0
    clean = bsq.orthogonalize(x.cuda())
    x[1, r, c] = bad
    got = bsq.orthogonalize(x.cuda())
    assert bool(got[1].isnan().all()), int((~got[1].isnan()).sum())
    assert torch.equal(got[0], clean[0]) and bool((got[2] == 0).all())
    # an update: the weights of its matrix, and the maximum over the stack
    w, m, g = (torch.stack([t, t, t]) for t in _update_case(shape, 5))
    ref = [t.clone().cuda() for t in (w, m)]
    bsq.muon_update(*ref, g.cuda(), 1e-2)
    wd, md = w.cuda(), m.cuda()
    md[1, r, c] = bad
    u = bsq.muon_update(wd, md, g.cuda(), 1e-2)
    assert bool(wd[1].isnan().all()) and bool(u["w_bf16"][1].isnan().all()) and bool(u["amax"].isnan().all())
    for i in (0, 2):
        assert torch.equal(wd[i], ref[0][i]) and torch.equal(md[i], ref[1][i])
    keep = torch.ones(R, C, dtype=torch.bool)
    keep[r, c] = False
    assert torch.equal(md[1].cpu()[keep], ref[1][1].cpu()[keep])


@pytest.mark.parametrize("shape", SHAPES[1:])
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e15, 1e30])
def test_sizes_of_values(shape, size):
    _check(_grad(shape, 6, size=size), eps=1e-37)


@pytest.mark.parametrize("shape", SHAPES[1:])
def test_large_epsilon(shape):
    _check(_grad(shape, 7), eps=1.0)                         # the norm is of the order of eps
    _check(_grad(shape, 7), eps=1e3)


@pytest.mark.parametrize("n", [200, 320, 577])
def test_permutation(n):
    """Singular values all equal, one entry a row: the other entries stay zero."""
    s = 1 / np.sqrt(n)
    for a, b, c in (bsq.NEWTON_SCHULZ,) * 5:
        s = a * s + b * s ** 3 + c * s ** 5
    p = torch.eye(n)[torch.randperm(n, generator=torch.Generator().manual_seed(8))] * 3.0
    got = bsq.orthogonalize(p.cuda()).double().cpu()
    assert torch.equal(got != 0, p != 0)
    # |p'| <= 3.45 per step: each rounding grows at most so, 4 roundings a step
    tol = sum(4 * 2.0 ** -11 * 3.45 ** k for k in range(5)) + 2.0 ** -8
    assert float((got[p != 0] / s - 1).abs().max()) <= tol


def _odd(t):
    """t at an address that only its type aligns."""
    return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [*SHAPES, (201, 333), (333, 201), (3, 301, 513)])
def test_out_strides_and_addresses(shape, dtype):
    announce("orthogonalize, addresses", shape, dtype)
    x = _grad(shape, 9, dtype).cuda()
    want = bsq.orthogonalize(x)
    guard = torch.full((x.numel() + 2,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[1:-1].view(shape)                            # 2-byte alignment only
    assert bsq.orthogonalize(x, out=out).data_ptr() == out.data_ptr() and torch.equal(out, want)
    assert float(guard[0]) == float(guard[-1]) == 7.0
    assert torch.equal(bsq.orthogonalize(x.mT.contiguous().mT), want)            # another memory order
    assert torch.equal(bsq.orthogonalize(_odd(x)), want)


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [*SHAPES, (201, 333), (333, 201), (3, 301, 513)])
def test_update_at_odd_addresses(shape, nesterov):
    announce("muon_update, addresses", shape)
    w, m, g = _update_case(shape, 10)
    want = _check_update(w, m, g, nesterov=nesterov)
    wo, mo, wb = _odd(w), _odd(m), _odd(g)
    u = bsq.muon_update(wo, mo, _odd(g), 1e-2, nesterov=nesterov, weight_decay=0.1, w_bf16=wb)
    assert torch.equal(wo, want[0]) and torch.equal(mo, want[1]) and torch.equal(u["w_bf16"], wo.bfloat16())
    assert u["w_bf16"].data_ptr() == wb.data_ptr() and float(u["amax"]) == float(wo.bfloat16().float().abs().max())


@pytest.mark.parametrize("shape", SHAPES)
def test_result_over_its_input_is_refused(shape):
    x = _grad(shape, 11, torch.bfloat16).cuda()
    x0 = x.clone()
    with pytest.raises(bsq.BsqError):
        bsq.orthogonalize(x, out=x)
    torch.cuda.synchronize()
    assert torch.equal(x, x0)
