"""Every kernel of the expert-grouped products by itself, against the oracle: the
library chooses by size, so each one is run here through the measurement library's
entry (libbsq's own launches) on ragged, empty and unassigned groups.  With dyadic
operands every FP32 partial sum is exact and the result must be the RNE of the
float64 one bit for bit; random operands use the GEMMs' stated tolerance."""

import ctypes
import os

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from oracle import gemm as OG
from oracle import moe as OM

from _gpu import announce, gpu
from test_gpu_grouped import BLK, _deq, _dev, _judge, _offsets, _operand

pytestmark = gpu

NAMES = ("direct 16x64", "direct 64x64", "direct 16x32", "lds 16x128", "lds 32x128", "lds 64x64", "lds 64x128",
         "lds 128x128", "256x256")
WGRAD_NAMES = ("direct 64x64", "lds 64x64", "lds 64x128", "lds 128x128", "256x256")
FMTS = ("nvfp4", "mxfp4", "mxfp8")


def grouped_on(name, wgrad, fmt, a, b, offsets, aa=None, ba=None, out=None):
    """bs_gemm_grouped[_wgrad] on the named kernel (None: the number of the chosen one)."""
    L = ctypes.CDLL(os.path.join(os.path.dirname(bsq.LIB_PATH), "libbsq_ceiling.so"))
    P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.bsq_grouped_on.argtypes = [I, I, I, I, P, I64, I64, I64, P, P, P, P, P, P, I, P, I64, P]
    E, K = len(offsets) - 1, a[0].shape[1] * (1 if fmt == "mxfp8" else 2)
    M, N = a[0].shape[0], b[0].shape[-2]
    if out is None:
        out = torch.full((E, M, N) if wgrad else (M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()
    v = -1 if name is None else NAMES.index(name)
    rc = L.bsq_grouped_on(v, int(wgrad), bsq.FORMATS[fmt], E, p(offsets), M, N, K, p(a[0]), p(a[1]), p(aa), p(b[0]),
                          p(b[1]), p(ba), 1 if ba is None else ba.numel(), p(out), N if wgrad else out.stride(0),
                          torch.cuda.current_stream().cuda_stream)
    if name is None:
        return rc
    assert rc == 0, (name, rc)
    return out


ROWS = [  # sizes, rows past the last group, N, K
    ([64, 1, 129, 0, 63], 7, 257, 512),
    ([257, 0, 511, 256, 3], 100, 520, 1024),
    ([1, 300], 0, 33, 1536),
]


def _rows_case(fmt, dyadic, sizes, past, N, K, seed=0):
    rng = np.random.default_rng(seed + N + K)
    E, R = len(sizes), sum(sizes) + past
    ac, asc = _operand(rng, R, K, fmt, dyadic)
    bc, bsc = _operand(rng, E * N, K, fmt, dyadic)
    am = np.array([2688.0], np.float32)
    bm = np.array([2688.0 * 2.0 ** (e % 3) for e in range(E)], np.float32) if dyadic else rng.uniform(1, 9, E).astype(np.float32)
    off = np.concatenate([[0], np.cumsum(sizes)])
    want, _ = OM.grouped(_deq(ac, asc, fmt), _deq(bc, bsc, fmt).reshape(E, N, K), off)
    if fmt == "nvfp4":
        for e in range(E):
            want[off[e]:off[e + 1]] *= OG.nvfp4_alpha(am[0], bm[e])
    ta, tb = _dev(am, bm) if fmt == "nvfp4" else (None, None)
    return _dev(ac, asc), _dev(bc.reshape(E, N, -1), bsc.reshape(E, N, -1)), ta, tb, want


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dyadic", [True, False])
@pytest.mark.parametrize("sizes,past,N,K", ROWS)
def test_rows(name, fmt, dyadic, sizes, past, N, K):
    announce("grouped rows on", name, fmt, dyadic, sizes, past, N, K)
    a, b, ta, tb, want = _rows_case(fmt, dyadic, sizes, past, N, K)
    out = torch.full((len(want), N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    grouped_on(name, False, fmt, a, b, _offsets(sizes), ta, tb, out[:, :N])
    _judge(out[:, :N], want, dyadic, (name, fmt, sizes, N, K))
    assert torch.all(out[:, N:] == 7), "wrote past the columns"
    whole = grouped_on(name, False, fmt, a, b, _offsets(sizes), ta, tb)
    assert torch.equal(whole, out[:, :N].contiguous())


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("fmt", FMTS)
def test_rows_whole_pieces_and_one_amax(name, fmt):
    """N % 8 == 0: the stores of whole 16-byte pieces; one amax for all experts."""
    announce("grouped rows on", name, fmt, "whole pieces")
    sizes, N, K = [70, 0, 330], 264, 512
    a, b, ta, _, _ = _rows_case(fmt, True, sizes, 3, N, K, 5)
    off = np.concatenate([[0], np.cumsum(sizes)])
    want, _ = OM.grouped(_deq(*(t.cpu().numpy() for t in a), fmt),
                         np.stack([_deq(*(t[e].cpu().numpy() for t in b), fmt) for e in range(3)]), off)
    _judge(grouped_on(name, False, fmt, a, b, _offsets(sizes), ta, ta), want, True, (name, fmt))


# groups in scale blocks of 16 (NVFP4) or 32 rows: starts and ends inside a K step,
# a pair and a period of every kernel; blocks past the last group
WGRAD = [
    ([3, 0, 5, 1, 40], 15, 100, 130),
    ([17, 15, 33, 31, 64, 0, 1, 95], 0, 260, 300),
    ([1, 30, 0, 1], 0, 257, 64),
]


def _wgrad_case(fmt, dyadic, blocks, past, M, N):
    rng = np.random.default_rng(len(blocks) * 10 + M + N)
    B = BLK[fmt]
    sizes = [v * B for v in blocks]
    R = -(-(sum(sizes) + past * B) // 512) * 512             # whole periods, so that every kernel takes them
    a, b = _operand(rng, M, R, fmt, dyadic), _operand(rng, N, R, fmt, dyadic)
    am, bm = np.float32(2688.0), np.float32(1344.0 if dyadic else 5.0)
    want, _ = OM.grouped_wgrad(_deq(*a, fmt), _deq(*b, fmt), np.concatenate([[0], np.cumsum(sizes)]))
    ta = tb = None
    if fmt == "nvfp4":
        want *= OG.nvfp4_alpha(am, bm)
        ta, tb = torch.tensor([am], device="cuda"), torch.tensor([bm], device="cuda")
    return _dev(*a), _dev(*b), sizes, ta, tb, want


@pytest.mark.parametrize("name", WGRAD_NAMES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dyadic", [True, False])
@pytest.mark.parametrize("blocks,past,M,N", WGRAD)
def test_wgrad(name, fmt, dyadic, blocks, past, M, N):
    announce("grouped wgrad on", name, fmt, dyadic, blocks, past, M, N)
    a, b, sizes, ta, tb, want = _wgrad_case(fmt, dyadic, blocks, past, M, N)
    got = grouped_on(name, True, fmt, a, b, _offsets(sizes), ta, tb)
    for e in range(len(blocks)):
        _judge(got[e], want[e], dyadic, (name, fmt, blocks, M, N, e))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("fmt", FMTS)
def test_rows_nan_stays_in_its_group(name, fmt):
    announce("grouped rows, NaN in one group, on", name, fmt)
    sizes, N, K = (40, 3, 270), 130, 512
    E, R, o = 3, sum(sizes) + 5, np.concatenate([[0], np.cumsum(sizes)])
    a, b, ta, tb, _ = _rows_case(fmt, False, sizes, 5, N, K, 22)
    run = lambda a, b: grouped_on(name, False, fmt, a, b, _offsets(sizes), ta, tb)
    want = run(a, b)
    assert torch.isfinite(want).all()
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    for bad in range(E):
        for which in (0, 1):
            sc = [a[1].clone(), b[1].clone()]
            if which == 0:
                sc[0][o[bad]:o[bad + 1]] = nan
            else:
                sc[1][bad] = nan
            got = run((a[0], sc[0]), (b[0], sc[1]))
            keep = torch.ones(R, dtype=torch.bool, device="cuda")
            keep[o[bad]:o[bad + 1]] = False
            assert torch.equal(got[keep], want[keep]) and torch.isnan(got[~keep]).all(), (bad, which)


@pytest.mark.parametrize("name", WGRAD_NAMES)
@pytest.mark.parametrize("fmt", FMTS)
def test_wgrad_nan_stays_in_its_group(name, fmt):
    announce("grouped wgrad, NaN in one group, on", name, fmt)
    blocks, M, N = (3, 21, 40), 130, 257
    B, per = BLK[fmt], 1 if fmt == "mxfp8" else 2
    a, b, sizes, ta, tb, _ = _wgrad_case(fmt, False, blocks, 2, M, N)
    o = np.concatenate([[0], np.cumsum(sizes)])
    K = a[0].shape[1] * per
    run = lambda a, b: grouped_on(name, True, fmt, a, b, _offsets(sizes), ta, tb)
    want = run(a, b)
    assert torch.isfinite(want).all()
    for bad in range(-1, len(blocks)):                       # -1: the rows past the last group
        k0, k1 = (o[bad], o[bad + 1]) if bad >= 0 else (o[-1], K)
        for which in (1, 2, 3):
            ops = []
            for i, (codes, scales) in enumerate((a, b)):
                codes, scales = codes.clone(), scales.clone()
                if which >> i & 1:
                    scales[:, k0 // B:k1 // B] = 0x7F if fmt == "nvfp4" else 0xFF
                    if fmt == "mxfp8":
                        codes[:, k0:k1] = 0x7F
                ops.append((codes, scales))
            got = run(*ops)
            for e in range(len(blocks)):
                if e != bad:
                    assert torch.equal(got[e], want[e]), (bad, which, e)
                else:
                    assert torch.isnan(got[e]).all(), (bad, which, e)


def _chosen(wgrad, fmt, E, rows, N, K):
    """The kernel of these sizes (rows spread evenly; nothing is computed)."""
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    z = torch.zeros(16, dtype=torch.uint8, device="cuda")
    per, B = (1 if fmt == "mxfp8" else 2), BLK[fmt]
    v = lambda *s: z.as_strided(s, (0,) * len(s))            # shapes and an aligned address only
    if wgrad:
        return NAMES[grouped_on(None, True, fmt, (v(N, rows // per), v(N, rows // B)), (v(K, rows // per), v(K, rows // B)), off,
                                out=v(1, 1))]
    return NAMES[grouped_on(None, False, fmt, (v(rows, K // per), v(rows, K // B)), (v(E, N, K // per), v(E, N, K // B)), off,
                            out=v(1, 1))]


def test_every_kernel_is_chosen_somewhere():
    """... by the library's own rule, at sizes of use: single tokens to training batches."""
    announce("the choice of grouped kernel")
    rows, wgrad = set(), set()
    for fmt in FMTS:
        for E in (2, 8, 64):
            for per in (1, 4, 16, 48, 128, 400, 2048):
                for N, K in ((256, 14336), (2048, 1408), (4096, 4096), (28672, 4096), (512, 512), (300, 96)):
                    rows.add(_chosen(False, fmt, E, per * E, N, K))
                    wgrad.add(_chosen(True, fmt, E, -(-per * E // 512) * 512, N, K))
        wgrad.add(_chosen(True, fmt, 4, 96, 256, 256))
    assert rows == set(NAMES) and wgrad == set(WGRAD_NAMES), (rows, wgrad)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("amax", [float("inf"), float("nan"), 0.0])
def test_rows_of_no_group_are_zero_whatever_the_amax(name, amax):
    """Rows past the last group are zeros, not 0 times an infinite decode scale, and
    no expert's amax reaches rows that are not its own."""
    announce("grouped rows, amax", amax, "on", name)
    sizes, N, K = (0, 20, 5), 130, 512
    a, b, ta, tb, _ = _rows_case("nvfp4", False, sizes, 40, N, K, 31)
    want = grouped_on(name, False, "nvfp4", a, b, _offsets(sizes), ta, tb)
    tb[0] = amax                                             # an expert without rows
    got = grouped_on(name, False, "nvfp4", a, b, _offsets(sizes), ta, tb)
    assert torch.equal(got, want) and torch.isfinite(want).all() and not want[25:].any()
    for bad in (ta, tb):                                     # everything that has a scale has this one
        bad.fill_(amax)
    got = grouped_on(name, False, "nvfp4", a, b, _offsets(sizes), ta, tb)
    assert not got[25:].any()
    if amax == float("inf"):                                 # its decode scale is infinite: the test tells
        assert not torch.isfinite(got[:25]).any()


@pytest.mark.parametrize("name", WGRAD_NAMES)
@pytest.mark.parametrize("amax", [float("inf"), float("nan")])
def test_wgrad_of_an_empty_group_is_zero_whatever_the_amax(name, amax):
    announce("grouped wgrad, amax", amax, "on", name)
    a, b, sizes, ta, tb, _ = _wgrad_case("nvfp4", False, (0, 5, 0, 30), 1, 130, 70)
    for bad in (ta, tb):
        keep = bad.clone()
        bad.fill_(amax)
        got = grouped_on(name, True, "nvfp4", a, b, _offsets(sizes), ta, tb)
        assert not got[0].any() and not got[2].any()
        if amax == float("inf"):
            assert not torch.isfinite(got[1]).any()
        bad.copy_(keep)


@pytest.mark.parametrize("amax", [float("inf"), float("nan")])
def test_products_without_a_reduction_are_zero_whatever_the_amax(amax):
    announce("grouped products without a reduction, amax", amax)
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    bad = torch.tensor([amax], device="cuda")
    out = torch.full((5, 9), 3.0, dtype=torch.bfloat16, device="cuda")
    bsq.bs_gemm_grouped("nvfp4", z(5, 0), z(5, 0), z(2, 9, 0), z(2, 9, 0), _offsets([2, 3]), bad, bad, out=out)
    assert not out.any()
    got = bsq.bs_gemm_grouped_wgrad("nvfp4", z(6, 0), z(6, 0), z(7, 0), z(7, 0), _offsets([0, 0]), bad, bad)
    assert got.shape == (2, 6, 7) and not got.any()


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("first", [1, 64, 300])
def test_rows_before_the_first_group_are_zero(name, fmt, first):
    """Offsets of some of the experts (one rank's, say) over the whole buffer: the rows
    before theirs belong to no group either."""
    announce("grouped rows, first group at", first, "on", name, fmt)
    sizes, past, N, K = [70, 0, 33], 20, 130, 512
    a, b, ta, tb, want = _rows_case(fmt, True, [first] + sizes, past, N, K, 41)
    off = _offsets([first] + sizes)
    b1 = tuple(t[1:].contiguous() for t in b)
    tb1 = None if tb is None else tb[1:].contiguous()
    want[:first] = 0
    _judge(grouped_on(name, False, fmt, a, b1, off[1:].contiguous(), ta, tb1), want, True, (name, fmt, first))
    none = torch.full((4,), sum(sizes) + first + past, dtype=torch.int32, device="cuda")     # no group has rows
    assert not grouped_on(name, False, fmt, a, b1, none, ta, tb1).any()
    got = bsq.bs_gemm_grouped(fmt, *a, *b1, off[1:].contiguous(), ta, tb1)
    _judge(got, want, True, (fmt, first))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("cancel", [False, True])
def test_mxfp8_sums_of_eight(name, cancel):
    """The stated error of MXFP8: 2^-13 of the largest of eight neighbouring products
    for each of them, the FP32 sum over K, and half a BF16 step; also where the large
    products cancel, in the same eight or in other ones."""
    announce("mxfp8 sums of eight on", name, cancel)
    rng = np.random.default_rng(51)
    R, N, K = 70, 130, 512
    ac, asc = _operand(rng, R, K, "mxfp8", False)
    bc, bsc = _operand(rng, N, K, "mxfp8", False)
    asc[:], bsc[:] = 127, 127
    if cancel:                                               # 256 * 256 - 256 * 256 in one eight and across two
        for i, j in ((0, 5), (40, 50), (300, 500)):
            ac[:, i], ac[:, j] = 0x78, 0xF8
            bc[:, i] = bc[:, j] = 0x78
    a, b = _deq(ac, asc, "mxfp8"), _deq(bc, bsc, "mxfp8")
    want, eights = a @ b.T, np.zeros((R, N))
    for g in range(0, K, 8):
        eights += np.abs(a[:, None, g:g + 8] * b[None, :, g:g + 8]).max(2)
    mag = np.abs(a) @ np.abs(b).T
    da, db = _dev(ac, asc), tuple(t[None] for t in _dev(bc, bsc))
    got = grouped_on(name, False, "mxfp8", da, db, _offsets([R])).double().cpu().numpy()
    # exact - got before the rounding: 8 products of each eight, K / 8 + 8 FP32 additions
    off = 8 * 2.0 ** -13 * eights + (K / 8 + 8) * 2.0 ** -24 * mag
    assert np.all(np.abs(got - want) <= off + 2.0 ** -8 * (np.abs(want) + off))
