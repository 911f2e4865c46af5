"""Integer codes hold no NaN: the scale of its row carries it, so that products, and a
training step, show it and do not go on from finite values.  Exact comparisons."""

import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from _gpu import announce, gpu
from fp8_quantized_gemm_amd.mlp import MLPLayer
from test_gpu_int8 import _acts, _codes

pytestmark = gpu

NAN, INF = float("nan"), float("inf")


def _same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16)) if a.dtype == torch.bfloat16 else torch.equal(a, b)


# rows in one wave, in a workgroup, in two passes; whole pieces and not
@pytest.mark.parametrize("cols", [8, 13, 256, 1000, 4096, 4097, 65536, 65537])
@pytest.mark.parametrize("bad", [NAN, -NAN, INF, -INF])
def test_quantize_rows(cols, bad):
    announce("int8_quantize, non-finite", cols, bad)
    x = _acts((6, cols), 1)
    c, s = bsq.int8_quantize(x.cuda())
    x[1, cols // 2], x[4, cols - 1] = bad, bad
    x[4, 0] = 3e38                                           # the largest finite value beside it
    d, t = bsq.int8_quantize(x.cuda())
    for r in (1, 4):
        assert bool(t[r].isnan()) if bad != bad else float(t[r]) == INF and bool((d[r] == 0).all())
    keep = [0, 2, 3, 5]
    assert torch.equal(d[keep], c[keep]) and torch.equal(t[keep], s[keep])


@pytest.mark.parametrize("shape", [(40, 64), (150, 129), (300, 520)])
def test_quantize_both(shape):
    """A value belongs to a row and to a column; the others' codes and scales stay."""
    announce("int8_quantize_transpose, non-finite", shape)
    R, C = shape
    x = _acts(shape, 2)
    p = bsq.int8_quantize_transpose(x.cuda())
    x[7, 5], x[R - 1, C - 2] = NAN, INF
    q = bsq.int8_quantize_transpose(x.cuda())
    assert bool(q["row_scales"][7].isnan()) and bool(q["col_scales"][5].isnan())
    assert float(q["row_scales"][R - 1]) == INF and float(q["col_scales"][C - 2]) == INF
    for side, bad, n in (("row", (7, R - 1), R), ("col", (5, C - 2), C)):
        keep = [i for i in range(n) if i not in bad]
        for k in (side + "_codes", side + "_scales"):
            assert torch.equal(q[k][keep], p[k][keep])


# one launch (few tokens, fewer and more pieces) and two; K off 16
@pytest.mark.parametrize("M,N,K", [(3, 50, 64), (5, 70, 2048), (40, 100, 512), (70, 130, 256), (200, 300, 1024), (6, 40, 1000)])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_linear(M, N, K, bad):
    announce("int8_linear, non-finite", M, N, K, bad)
    x = _acts((M, K), 3)
    w, sw = (t.cuda() for t in _codes((N, K), 4))
    bias = torch.randn(N, device="cuda")
    clean = bsq.int8_linear(x.cuda(), w, sw, bias)
    x[1, K - 1] = bad
    x[1, 0] = 0
    y = bsq.int8_linear(x.cuda(), w, sw, bias)
    assert bool(y[1].isnan().all())
    keep = [i for i in range(M) if i != 1]
    assert _same_bits(y[keep], clean[keep])


def test_training_step_shows_it():
    """A NaN in dY reaches the input's gradient and the weights' gradients."""
    announce("MLPLayer int8, NaN in dY")
    g = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(s, generator=g)
    L = MLPLayer((0.05 * rn(96, 64)).cuda(), (0.05 * rn(64, 48)).cuda(), 32, fmt="int8")
    x, dy = rn(32, 64).bfloat16().cuda(), (1e-2 * rn(32, 64)).bfloat16()
    dy[3, 9] = NAN
    L.forward(x)
    dx = L.backward(dy.cuda())
    assert bool(dx[3].isnan().all()) and bool(L.grad["W_down"][9].isnan().all()) and bool(L.grad["W_gu"].isnan().any())
    L.update()
    assert bool(L.w32["W_down"][9].isnan().all())
