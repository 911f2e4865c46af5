"""Orthogonalisation of matrices of every rank against the FP64 definition, to the accuracy
that include/bsq.h states.  The result is read in FP32 out of an update of zero weights (the
momentum is the matrix: mu 1, a zero gradient; lr and scale 1), so that no output rounding
hides it; products pass it to the update in FP16, which adds 2^-11 of its norm."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from _gpu import announce, gpu
from muon_matrices import distance, matrices, stated
from oracle import muon as OM

pytestmark = gpu


def _orthogonal(x, steps):
    """What muon_update subtracts for the momentum x [R, C] (FP32), as FP64."""
    w, m = torch.zeros(x.shape, device="cuda"), x.cuda()
    bsq.muon_update(w, m, torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda"), 1.0, mu=1.0, nesterov=False, scale=1.0,
                    steps=steps)
    assert torch.equal(m.cpu(), x)
    return -w.double().cpu().numpy()


# one workgroup of each width; products, single steps and pairs, wide and tall
@pytest.mark.parametrize("steps", [5, 8])
@pytest.mark.parametrize("shape", [(2, 3), (16, 16), (16, 24), (32, 1024), (768, 64), (96, 500), (128, 256), (250, 160),
                                   (64, 1300), (200, 330), (330, 200), (320, 320), (320, 512), (700, 300), (512, 1024)])
def test_any_rank(shape, steps):
    announce("muon_update, ranks", shape, steps)
    for name, x in matrices(*shape, seed=3):
        t = torch.from_numpy(x).float()
        e = OM.orthogonalize(t.double().numpy(), steps=steps)
        d = distance(_orthogonal(t, steps), e)
        assert d <= stated(*shape, steps) + 2.0 ** -11, (shape, steps, name, d)


@pytest.mark.parametrize("shape,rank", [((1408, 2048), 1), ((1408, 2048), 176), ((1408, 2048), 469), ((2048, 2048), 1),
                                        ((2048, 2048), 682), ((4096, 1024), 341)])
def test_sizes_of_layers(shape, rank):
    """Rank 1, m / 8 and m / 3 (where pairs of steps are furthest off)."""
    announce("muon_update, rank", shape, rank)
    g = torch.Generator().manual_seed(5)
    t = torch.randn(shape[0], rank, generator=g) @ torch.randn(rank, shape[1], generator=g)
    d = distance(_orthogonal(t, 5), OM.orthogonalize(t.double().numpy()))
    assert d <= stated(*shape) + 2.0 ** -11, d


@pytest.mark.parametrize("shape", [(64, 128), (200, 330), (320, 512)])
def test_one_token(shape):
    """A weight's gradient after one token (rank 1), through orthogonalize and its BF16 output."""
    announce("orthogonalize, one token", shape)
    g = torch.Generator().manual_seed(4)
    dy, x = torch.randn(shape[0], 1, generator=g).bfloat16(), torch.randn(1, shape[1], generator=g).bfloat16()
    grad = (dy.float() @ x.float())
    e = OM.orthogonalize(grad.double().numpy())
    y = bsq.orthogonalize(grad.cuda()).double().cpu().numpy()
    assert distance(y, e) <= stated(*shape) + 2.0 ** -8
