"""8-bit integer quantizers and products against the oracle, bit for bit: every step
of the definition is one FP32 rounding and the sums are integers, so there is no
tolerance."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from _gpu import announce, bits, f32, gpu
from oracle import int8 as OI

pytestmark = gpu


def _acts(shape, seed, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if outliers:
        x = torch.where(torch.rand(shape, generator=g) < 1e-2, 50 * x, x)
    x = x * torch.exp(torch.randn((shape[0], 1), generator=g))
    if shape[0] > 2:
        x[2] = 0
    return x.bfloat16()


def _codes(shape, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
    s = torch.rand(shape[0], generator=g) * 0.1 + 1e-3
    return c, s


def _same(got, want, what):
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape, what
    bad = np.argwhere(got != want)
    assert len(bad) == 0, (what, len(bad), bad[:3].tolist(), got[tuple(bad[0])], want[tuple(bad[0])])


SHAPES = [(1, 1), (1, 16), (3, 7), (5, 8), (4, 130), (63, 512), (9, 513), (7, 1024), (6, 2048), (3, 2049), (5, 4096), (2, 8200),
          (3, 16384), (2, 16392), (2, 14337), (1, 65536), (2, 65537), (1025, 24)]


@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_rows(shape):
    announce("int8_quantize", shape)
    x = _acts(shape, 1)
    c, s = bsq.int8_quantize(x.cuda())
    oc, os_ = OI.quantize(bits(x))
    _same(s.cpu(), os_, "scales")
    _same(c.cpu(), oc, "codes")


@pytest.mark.parametrize("shape", [(1, 1), (1, 24), (24, 1), (16, 16), (7, 9), (128, 128), (129, 130), (255, 520), (256, 512),
                                   (257, 1032), (300, 514), (1000, 136), (33, 4096), (1027, 1025)])
def test_quantize_both(shape):
    announce("int8_quantize_transpose", shape)
    x = _acts(shape, 2)
    q = bsq.int8_quantize_transpose(x.cuda())
    for side, y in (("row", x), ("col", x.t().contiguous())):
        oc, os_ = OI.quantize(bits(y))
        _same(q[side + "_scales"].cpu(), os_, side + " scales")
        _same(q[side + "_codes"].cpu(), oc, side + " codes")
    for side in ("row", "col"):
        p = bsq.int8_quantize_transpose(x.cuda(), row=side == "row", col=side == "col")
        _same(p[side + "_codes"].cpu(), q[side + "_codes"].cpu(), side + " alone")
        assert p[("col" if side == "row" else "row") + "_codes"] is None


def test_quantize_extremes():
    x = torch.tensor([[2.0 ** -133, 0, -2.0 ** -133, 0], [3e38, -1e38, 1e-38, 0], [0, 0, 0, 0], [-0.0, 1.5, -2.5, 127]]).bfloat16()
    c, s = bsq.int8_quantize(x.cuda())
    oc, os_ = OI.quantize(bits(x))
    _same(c.cpu(), oc, "codes")
    _same(s.cpu(), os_, "scales")


def test_non_finite_stays_in_its_row():
    x = _acts((8, 256), 3)
    y = x.clone()
    y[5, 17], y[6, 3] = float("nan"), float("inf")
    c, s = bsq.int8_quantize(x.cuda())
    d, t = bsq.int8_quantize(y.cuda())
    keep = [0, 1, 2, 3, 4, 7]
    _same(d.cpu()[keep], c.cpu()[keep], "codes")
    _same(t.cpu()[keep], s.cpu()[keep], "scales")


def _check_gemm(M, N, K, bias=False, ldc=None, seed=5):
    a, sa = _codes((M, K), seed)
    b, sb = _codes((N, K), seed + 1)
    bi = torch.randn(N, generator=torch.Generator().manual_seed(seed + 2)) if bias else None
    out = None
    if ldc:
        buf = torch.full((M, ldc), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:, :N]
    got = bsq.int8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), bias=None if bi is None else bi.cuda(), out=out)
    want = OI.gemm(a.numpy(), sa.numpy(), b.numpy(), sb.numpy(), None if bi is None else bi.numpy())
    _same(f32(got).astype(np.float64), want, (M, N, K))
    if ldc:
        assert bool((buf[:, N:] == 7.0).all()), "columns past N were written"


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 1, 15), (1, 5, 16), (2, 3, 17), (1, 64, 128), (1, 200, 129), (5, 33, 63), (16, 64, 256), (17, 65, 255),
    (16, 70, 1000), (33, 31, 144), (64, 64, 64), (65, 63, 200), (100, 300, 512), (128, 128, 640), (129, 257, 384),
    (255, 256, 1408), (256, 256, 2048), (257, 513, 528), (300, 700, 4096), (511, 100, 1031), (513, 1025, 1024), (1, 4096, 4096),
    (37, 2048, 1408), (640, 640, 112)])
@pytest.mark.parametrize("bias", [False, True])
def test_gemm(M, N, K, bias):
    announce("int8_gemm", M, N, K, bias)
    _check_gemm(M, N, K, bias)


@pytest.mark.parametrize("M,N,K,ldc", [(3, 5, 32, 8), (70, 130, 256, 133), (300, 520, 384, 528)])
def test_gemm_strided_output(M, N, K, ldc):
    announce("int8_gemm ldc", M, N, K, ldc)
    _check_gemm(M, N, K, True, ldc)


def test_gemm_no_reduction():
    """K = 0: the bias, or zeros."""
    a, b = torch.empty(3, 0, dtype=torch.int8, device="cuda"), torch.empty(5, 0, dtype=torch.int8, device="cuda")
    bias = torch.tensor([1.0, -2, 3, 0.5, 0], device="cuda")
    s3, s5 = torch.ones(3, device="cuda"), torch.ones(5, device="cuda")
    assert torch.equal(bsq.int8_gemm(a, s3, b, s5, bias=bias), bias.bfloat16().expand(3, 5))
    assert torch.equal(bsq.int8_gemm(a, s3, b, s5), torch.zeros(3, 5, dtype=torch.bfloat16, device="cuda"))


def test_gemm_largest_sums():
    """The longest reduction of the largest codes stays in 32 bits: K 131,071 of -128 x -128."""
    K = 131071
    a = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((70, K), -128, dtype=torch.int8, device="cuda")
    b[1:] = 127
    one = torch.ones(70, device="cuda")
    got = bsq.int8_gemm(a, one[:2], b, one)
    want = torch.tensor([128.0 * 128 * K, -128.0 * 127 * K]).float().bfloat16()
    assert torch.equal(got[:, 0].cpu(), want[:1].expand(2)) and torch.equal(got[:, 1:].cpu(), want[1:].expand(2, 69))


def test_zero_sizes():
    z = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    c, s = bsq.int8_quantize(z(0, 16))
    assert c.shape == (0, 16) and s.shape == (0,)
    c, s = bsq.int8_quantize(z(3, 0))
    assert c.shape == (3, 0) and torch.equal(s, torch.ones(3, device="cuda"))
    q = bsq.int8_quantize_transpose(z(0, 5))
    assert q["col_codes"].shape == (5, 0) and torch.equal(q["col_scales"], torch.ones(5, device="cuda"))
    w, sw = torch.zeros(8, 16, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    assert bsq.int8_linear(z(0, 16), w, sw).shape == (0, 8)
    assert bsq.int8_linear(torch.ones(2, 16, device="cuda").bfloat16(), w[:0], sw[:0]).shape == (2, 0)


# few rows (one launch): each number of waves per row, of row tiles and of column tiles,
# K below, at and off whole groups, the most codes; then the two launches
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (1, 12300, 8192), (1, 5, 16), (2, 64, 32), (2, 6200, 2064), (3, 100, 144),
                                   (4, 20, 8192), (5, 33, 496), (8, 1000, 2048), (8, 70, 8192), (15, 12288, 528),
                                   (16, 2048, 1408), (16, 77, 4096), (17, 300, 112), (31, 6150, 640), (32, 50, 2048),
                                   (33, 90, 256), (37, 2048, 1408), (48, 6144, 1264), (64, 129, 1024), (63, 1, 128),
                                   (65, 129, 1024), (64, 257, 1040), (1, 300, 1000), (2, 64, 24), (64, 257, 513), (9, 30, 8208),
                                   (200, 512, 4096), (700, 1024, 1536)])
@pytest.mark.parametrize("bias", [False, True])
def test_linear(M, N, K, bias):
    announce("int8_linear", M, N, K, bias)
    x = _acts((M, K), 7)
    w, sw = _codes((N, K), 8)
    b = torch.randn(N, generator=torch.Generator().manual_seed(9)) if bias else None
    got = bsq.int8_linear(x.cuda(), w.cuda(), sw.cuda(), bias=None if b is None else b.cuda())
    c, s = OI.quantize(bits(x))
    _same(f32(got).astype(np.float64), OI.gemm(c, s, w.numpy(), sw.numpy(), None if b is None else b.numpy()), (M, N, K))


def test_out_argument_and_strided_input():
    x = _acts((40, 96), 11).cuda()
    w, sw = (t.cuda() for t in _codes((24, 48), 12))
    want = bsq.int8_linear(x[:, :48].contiguous(), w, sw)
    buf = torch.zeros(40, 32, dtype=torch.bfloat16, device="cuda")
    got = bsq.int8_linear(x[:, :48], w, sw, out=buf[:, :24])
    assert torch.equal(got, want) and got.data_ptr() == buf.data_ptr() and bool((buf[:, 24:] == 0).all())
    with pytest.raises(ValueError):
        bsq.int8_linear(x[:, :48], w, sw, out=torch.zeros(40, 23, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        bsq.int8_gemm(w.t(), sw, w, sw)
    with pytest.raises(bsq.BsqError):                        # 2^17 products do not fit the sums
        big = torch.zeros(1, 1 << 17, dtype=torch.int8, device="cuda")
        bsq.int8_gemm(big, sw[:1], big, sw[:1])


def test_offsets_past_32_bits():
    """Operands and outputs above 4 GiB: rows at the far end against the same rows by themselves."""
    M, N, K = 140000, 16384, 32
    announce("int8_gemm large", M, N, K)
    a, sa = (t.cuda() for t in _codes((M, K), 13))
    b, sb = (t.cuda() for t in _codes((N, K), 14))
    big = bsq.int8_gemm(a, sa, b, sb)                        # 4.6 GB
    for rows in (slice(0, 64), slice(131072, 131172), slice(M - 100, M)):
        assert torch.equal(big[rows], bsq.int8_gemm(a[rows].contiguous(), sa[rows].contiguous(), b, sb))
    del big
    K2 = 131056
    b2 = torch.randint(-127, 128, (33000, K2), dtype=torch.int8, device="cuda")       # 4.3 GB
    s2 = torch.rand(33000, device="cuda")
    a2, sa2 = (t.cuda() for t in _codes((3, K2), 15))
    far = bsq.int8_gemm(a2, sa2, b2, s2)
    assert torch.equal(far[:, 32900:], bsq.int8_gemm(a2, sa2, b2[32900:].contiguous(), s2[32900:].contiguous()))


def test_streams_and_graph():
    """On another stream; captured, replayed several times with eager work between the
    replays, on inputs that change."""
    x = _acts((33, 512), 16).cuda()
    w, sw = (t.cuda() for t in _codes((200, 512), 17))
    other = _acts((300, 384), 18).cuda()
    want = bsq.int8_linear(x, w, sw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = bsq.int8_linear(x, w, sw)
    s.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = bsq.int8_linear(x, w, sw)
        q = bsq.int8_quantize_transpose(other)
    for i in range(4):
        x.copy_(_acts((33, 512), 20 + i))
        other.copy_(_acts((300, 384), 30 + i))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bsq.int8_linear(x, w, sw))
        e = bsq.int8_quantize_transpose(other)
        assert all(torch.equal(q[k], e[k]) for k in q)
