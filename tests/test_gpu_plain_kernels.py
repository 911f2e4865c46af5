"""Each kernel of the plain products by itself, through the measurement library: the
8-bit integer products bit for bit, the orthogonalisation's FP16 products on every
kernel against the FP64 definition (the tolerance of test_gpu_muon)."""

import ctypes
import os

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from _gpu import announce, f32, gpu
from oracle import int8 as OI
from oracle import muon as OM
from test_gpu_int8 import _codes, _same
from test_gpu_muon import _allowed, _grad

pytestmark = gpu + [pytest.mark.skipif(not os.path.exists(os.path.join(bsq._PKG, "libbsq_ceiling.so")),
                                       reason="libbsq_ceiling.so not built")]

DIRECT16, DIRECT64, RING128, RING192, RING256, RING128X5, RING64, RING96 = range(8)
RINGS = (RING64, RING96, RING128, RING128X5, RING192, RING256)


@pytest.fixture(scope="module")
def lib():
    bsq.lib()
    L = ctypes.CDLL(os.path.join(bsq._PKG, "libbsq_ceiling.so"))
    P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    L.bsq_int8_on.argtypes = [I, I, I, I64, I64, I64, P, P, P, P, P, P, I64, P]
    L.bsq_ortho_on.argtypes = [I, I, P, I, I64, I64, I64, I, P, F, P, P, P]
    return L


def _int8_on(L, kernel, M, N, K, a, sa, b, sb, bias, out, rest=-1, count=0):
    return L.bsq_int8_on(kernel, rest, count, M, N, K, a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(),
                         None if bias is None else bias.data_ptr(), out.data_ptr(), out.stride(0),
                         torch.cuda.current_stream().cuda_stream)


# K: one unit and less, one more and one less than the rings' buffers, ends in every chunk
SIZES = [(64, 64, 16), (256, 256, 128), (1, 1, 112), (257, 255, 144), (300, 130, 256), (129, 513, 384), (200, 200, 400),
         (512, 300, 512), (256, 384, 640), (130, 257, 656), (255, 640, 768), (384, 192, 896), (100, 100, 1040), (640, 520, 2048)]


# a kernel by itself, or (kernel, the smaller one that the tiles from a number on are cut for, that number)
CUTS = [(RING256, RING128, 1), (RING256, RING64, 2), (RING256, RING128X5, 0), (RING192, RING96, 1), (RING192, RING64, 3),
        (RING128, RING64, 2), (RING128X5, RING64, 1)]


@pytest.mark.parametrize("kernel", [DIRECT16, DIRECT64, *RINGS, *CUTS])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_int8(lib, kernel, M, N, K):
    announce("int8 kernel", kernel, M, N, K)
    kernel, rest, count = kernel if isinstance(kernel, tuple) else (kernel, -1, 0)
    side = {RING256: 256, RING192: 192}.get(kernel, 128)
    if rest >= 0:
        count = min(count, -(-M // side) * -(-N // side) - 1)
    a, sa = _codes((M, K), M)
    b, sb = _codes((N, K), N)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(K))
    out = torch.full((M + 1, N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    dev = [t.cuda() for t in (a, sa, b, sb, bias)]
    assert _int8_on(lib, kernel, M, N, K, *dev, out, rest, count) == 0
    torch.cuda.synchronize()
    want = OI.gemm(a.numpy(), sa.numpy(), b.numpy(), sb.numpy(), bias.numpy())
    _same(f32(out[:M, :N]).astype(np.float64), want, (kernel, M, N, K))
    assert bool((out[M:] == 7.0).all()) and bool((out[:, N:] == 7.0).all()), "written outside the output"


def test_int8_refused(lib):
    """The rings take whole 16-byte chunks only."""
    a, s = torch.zeros(64, 24, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    out = torch.full((64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for k in (*RINGS, 99):
        assert _int8_on(lib, k, 64, 64, 24, a, s, a, s, None, out) == -1
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("kernel", [*RINGS, *CUTS])
@pytest.mark.parametrize("shape", [(64, 64), (1, 100, 60), (2, 200, 136), (3, 130, 400), (1, 520, 500), (1, 300, 1000), (1, 1000, 257)])
def test_ortho(lib, kernel, shape):
    announce("ortho kernel", kernel, shape)
    x = _grad(shape, 9)
    xs = x.cuda()
    B, R, C = shape if len(shape) == 3 else (1, *shape)
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((bsq._size("orthogonalize_workspace", B, R, C),), 0xFF, dtype=torch.uint8, device="cuda")
    coefs = bsq._coefs(5, OM.COEFS)
    k, rest = kernel[:2] if isinstance(kernel, tuple) else (kernel, -1)
    assert lib.bsq_ortho_on(k, rest, xs.data_ptr(), 1, B, R, C, 5, coefs, 1e-7, out.data_ptr(), ws.data_ptr(),
                            torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for m, y in zip(x.double().reshape(B, R, C).numpy(), out.double().cpu().reshape(B, R, C).numpy()):
        e = OM.orthogonalize(m)
        err, tol = np.linalg.norm(y - e), _allowed(m, e, 5, OM.COEFS, 1e-7, 2.0 ** -8,
                                                 OM.phases(*sorted((v + 63) // 64 * 64 for v in m.shape), 5))
        assert err <= tol, (kernel, shape, err, tol)
