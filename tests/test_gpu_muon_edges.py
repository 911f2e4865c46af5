"""The orthogonalisation and its update where the values are extreme, in both forms: one
workgroup, single steps by products, and pairs of steps by products.  Tolerances are
those of test_gpu_muon."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from _gpu import announce, gpu
from test_gpu_muon import _check, _grad

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
