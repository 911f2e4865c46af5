"""Expert-grouped products against the oracle.  With dyadic operands (unit or
power-of-two scales, few significant bits) every FP32 partial sum is exact, so the
result must be the RNE of the float64 one bit for bit; random operands use the
GEMMs' stated tolerance (oracle.gemm.tolerance_report)."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from oracle import formats as F
from oracle import gemm as OG
from oracle import moe as OM

from _gpu import announce, gpu

pytestmark = gpu

BLK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}


def _operand(rng, rows, K, fmt, dyadic):
    """codes, scales (numpy uint8)."""
    if fmt == "mxfp8":
        if dyadic:
            codes = (rng.integers(0, 2, (rows, K)) << 7 | rng.integers(0x38, 0x50, (rows, K))).astype(np.uint8)
        else:
            codes = (rng.integers(0, 2, (rows, K)) << 7 | rng.integers(0x20, 0x7F, (rows, K))).astype(np.uint8)
    else:
        codes = rng.integers(0, 256, (rows, K // 2)).astype(np.uint8)
    shape = (rows, K // BLK[fmt])
    if fmt == "nvfp4":
        scales = rng.choice([0x38, 0x40, 0x48], shape) if dyadic else rng.integers(1, 0x7F, shape)
    else:
        scales = rng.integers(126, 129, shape) if dyadic else rng.integers(118, 130, shape)
    return codes, scales.astype(np.uint8)


def _deq(codes, scales, fmt):
    return OG.dequant_nvfp4(codes, scales) if fmt == "nvfp4" else OG.dequant_mx(codes, scales, fmt)


def _dev(*a):
    return tuple(torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in a)


def _offsets(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def _judge(got, want, dyadic, what):
    got = got.double().cpu().numpy()
    if dyadic:
        assert np.array_equal(got, F.f64_to_bf16_rne(want)), (what, int(np.sum(got != F.f64_to_bf16_rne(want))))
    else:
        rep = OG.tolerance_report(got, want)
        assert rep["passed"], (what, rep)


ROWS = [  # sizes, rows past the last group, N, K
    ([1], 0, 1, 32),
    ([0, 1, 0], 0, 64, 64),
    ([2, 0, 0, 3, 1, 0, 0, 0], 2, 100, 128),
    ([16, 17, 15], 0, 130, 160),
    ([0, 0, 70, 5], 53, 64, 96),
    ([64, 1, 129, 0, 63], 7, 257, 512),
    ([5] * 70, 0, 72, 256),
    ([33, 200], 31, 65, 1408),
    ([300], 0, 300, 544),
    ([257, 0, 511, 256, 3], 100, 520, 1024),
    ([180] * 67 + [0, 1, 700], 300, 40, 256),
    ([1, 1023, 0, 2], 0, 33, 768),
    ([40, 70, 33, 0, 90], 10, 150, 320),
    ([64, 65, 63, 128, 1], 0, 129, 640),
    ([130, 127, 90], 70, 260, 384),
    ([40, 41, 39], 0, 128, 192),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dyadic", [True, False])
@pytest.mark.parametrize("sizes,past,N,K", ROWS)
def test_rows(fmt, dyadic, sizes, past, N, K):
    announce("bs_gemm_grouped", fmt, dyadic, sizes[:8], past, N, K)
    rng = np.random.default_rng(len(sizes) * 100 + N + K)
    E, R = len(sizes), sum(sizes) + past
    ac, asc = _operand(rng, R, K, fmt, dyadic)
    bc, bsc = _operand(rng, E * N, K, fmt, dyadic)
    # amax 2688: decode scale exactly 1
    am = np.array([2688.0], np.float32)
    bm = np.array([2688.0 * 2.0 ** (e % 3) for e in range(E)], np.float32) if dyadic else rng.uniform(1, 9, E).astype(np.float32)
    off = np.concatenate([[0], np.cumsum(sizes)])
    want, _ = OM.grouped(_deq(ac, asc, fmt), _deq(bc, bsc, fmt).reshape(E, N, K), off)
    if fmt == "nvfp4":
        for e in range(E):
            want[off[e]:off[e + 1]] *= OG.nvfp4_alpha(am[0], bm[e])
    tac, tas, tbc, tbs = _dev(ac, asc, bc.reshape(E, N, -1), bsc.reshape(E, N, -1))
    ta, tb = _dev(am, bm)
    nv = fmt == "nvfp4"
    out = torch.full((R, N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    bsq.bs_gemm_grouped(fmt, tac, tas, tbc, tbs, _offsets(sizes), ta if nv else None, tb if nv else None, out=out[:, :N])
    _judge(out[:, :N], want, dyadic, (fmt, sizes[:8], N, K))
    assert torch.all(out[:, N:] == 7), "wrote past the columns"
    got = bsq.bs_gemm_grouped(fmt, tac, tas, tbc, tbs, _offsets(sizes), ta if nv else None, tb if nv else None)
    assert torch.equal(got, out[:, :N].contiguous())


def _bits(shape, fmt, seed):
    """Random finite codes of any amount, made on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 0x7F if fmt == "mxfp8" else 256, shape, dtype=torch.uint8, device="cuda", generator=g)


@pytest.mark.parametrize("fmt,E,N,K", [("nvfp4", 130, 8192, 8192), ("mxfp4", 130, 8192, 8192), ("mxfp8", 66, 8192, 8192)])
def test_rows_with_weights_past_32_bit_offsets(fmt, E, N, K):
    """Weights of more than 4 GiB: the last expert's products are those of the
    expert alone, whatever kernel either size takes (every partial sum is exact)."""
    announce("bs_gemm_grouped, weights past 4 GiB", fmt)
    rng = np.random.default_rng(11)
    sizes = [0] * E
    sizes[0], sizes[E // 2], sizes[E - 1] = 3, 1, 40
    ac, asc = _dev(*_operand(rng, 44, 64, fmt, True))
    a = torch.zeros((44, K if fmt == "mxfp8" else K // 2), dtype=torch.uint8, device="cuda")
    a[:, -ac.shape[1]:] = ac                                 # the last 64 elements only: exact sums
    unit = 0x38 if fmt == "nvfp4" else 127
    asc = torch.full((44, K // BLK[fmt]), unit, dtype=torch.uint8, device="cuda")
    b = _bits((E, N, a.shape[1]), fmt, 12)
    b[:, :, -ac.shape[1]:] &= 0xBF if fmt == "mxfp8" else 0xFF
    bs = torch.full((E, N, K // BLK[fmt]), unit, dtype=torch.uint8, device="cuda")
    am = torch.tensor([2688.0], device="cuda") if fmt == "nvfp4" else None
    got = bsq.bs_gemm_grouped(fmt, a, asc, b, bs, _offsets(sizes), am, am)
    r = 0
    for e, n in ((0, 3), (E // 2, 1), (E - 1, 40)):
        tail = lambda t, d: np.ascontiguousarray(t[..., -d:].cpu().numpy())
        d, sd = ac.shape[1], 64 // BLK[fmt]
        want = _deq(tail(a[r:r + n], d), tail(asc[r:r + n], sd), fmt) @ _deq(tail(b[e], d), tail(bs[e], sd), fmt).T
        _judge(got[r:r + n], want, fmt != "mxfp8", (fmt, e))
        r += n


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_reductions_of_more_than_2_24(fmt):
    """Rows of 2^24 + 64 elements (64-bit offsets inside a tile): ones at both ends
    and in the middle of K, by small whole numbers."""
    announce("grouped products, K past 2^24", fmt)
    K = (1 << 24) + 64
    rng = np.random.default_rng(13)
    at = np.array([0, 1, K // 2, K - 33, K - 1])
    one = {"nvfp4": 2, "mxfp4": 2, "mxfp8": 0x38}[fmt]       # the code of 1.0
    val = {"nvfp4": [2, 4, 6], "mxfp4": [2, 4, 6], "mxfp8": [0x38, 0x40, 0x48]}[fmt]      # 1, 2, 4

    def sparse(rows, pick):
        t = torch.zeros((rows, K if fmt == "mxfp8" else K // 2), dtype=torch.uint8, device="cuda")
        v = np.zeros((rows, len(at)))
        for r in range(rows):
            for i, k in enumerate(at):
                c = pick()
                v[r, i] = 1.0 if c == one else 2.0 ** (val.index(c))
                if fmt == "mxfp8":
                    t[r, k] = c
                else:
                    t[r, k // 2] += c << (4 * (int(k) & 1))
        s = torch.full((rows, K // BLK[fmt]), 0x38 if fmt == "nvfp4" else 127, dtype=torch.uint8, device="cuda")
        return t, s, v
    a, asc, av = sparse(5, lambda: one)
    b, bsc, bv = sparse(6, lambda: int(rng.choice(val)))
    am = torch.tensor([2688.0], device="cuda") if fmt == "nvfp4" else None
    got = bsq.bs_gemm_grouped(fmt, a, asc, b.view(2, 3, -1), bsc.view(2, 3, -1), _offsets([4, 1]), am, am)
    want = np.concatenate([av[:4] @ bv[:3].T, av[4:] @ bv[3:].T])
    _judge(got, want, True, fmt)
    cut = K // 2 // 32 * 32
    got = bsq.bs_gemm_grouped_wgrad(fmt, a, asc, b, bsc, _offsets([cut, K - cut]), am, am)
    lo = at < cut
    want = np.stack([av[:, lo] @ bv[:, lo].T, av[:, ~lo] @ bv[:, ~lo].T])
    _judge(got, want, True, fmt)


def test_rows_nvfp4_half_block_and_shared_amax():
    announce("bs_gemm_grouped nvfp4 K = 16, 48, 272, one amax")
    rng = np.random.default_rng(1)
    for K in (16, 48, 272):
        sizes, N = [3, 0, 40], 33
        ac, asc = _operand(rng, 43, K, "nvfp4", True)
        bc, bsc = _operand(rng, 3 * N, K, "nvfp4", True)
        one = torch.tensor([2688.0], device="cuda")
        want, _ = OM.grouped(_deq(ac, asc, "nvfp4"), _deq(bc, bsc, "nvfp4").reshape(3, N, K), [0, 3, 3, 43])
        tac, tas, tbc, tbs = _dev(ac, asc, bc.reshape(3, N, -1), bsc.reshape(3, N, -1))
        _judge(bsq.bs_gemm_grouped("nvfp4", tac, tas, tbc, tbs, _offsets(sizes), one, one), want, True, K)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_rows_without_a_reduction_are_zero(fmt):
    announce("bs_gemm_grouped K = 0", fmt)
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    out = torch.full((5, 9), 3.0, dtype=torch.bfloat16, device="cuda")
    bsq.bs_gemm_grouped(fmt, z(5, 0), z(5, 0), z(2, 9, 0), z(2, 9, 0), _offsets([2, 3]), one, one, out=out)
    assert not out.any()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_rows_with_offsets_past_the_rows(fmt):
    """Offsets outside [0, rows] are read as the nearest bound."""
    announce("bs_gemm_grouped clamped offsets", fmt)
    rng = np.random.default_rng(2)
    ac, asc = _operand(rng, 20, 64, fmt, True)
    bc, bsc = _operand(rng, 2 * 40, 64, fmt, True)
    tac, tas, tbc, tbs = _dev(ac, asc, bc.reshape(2, 40, -1), bsc.reshape(2, 40, -1))
    one = torch.tensor([2688.0], device="cuda")
    f = lambda o: bsq.bs_gemm_grouped(fmt, tac, tas, tbc, tbs, torch.tensor(o, dtype=torch.int32, device="cuda"), one, one)
    assert torch.equal(f([-4, 7, 1 << 30]), f([0, 7, 20]))


WGRAD = [  # sizes (in scale blocks), blocks past the last group, M, N
    ([1], 0, 1, 1),
    ([0, 2, 0], 1, 64, 33),
    ([3, 0, 5, 1], 0, 100, 130),
    ([8, 16, 40, 0], 16, 65, 257),
    ([17, 15, 33, 31, 64, 0, 1, 95], 0, 256, 300),
    ([100, 1, 27], 128, 520, 264),
    ([5, 6, 1, 100, 0, 2, 142], 0, 300, 40),
    ([1, 510, 0, 1], 0, 257, 64),
    ([7, 1, 3, 9, 0, 2, 2], 0, 140, 129),
    ([3, 4, 1, 4], 4, 70, 260),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dyadic", [True, False])
@pytest.mark.parametrize("blocks,past,M,N", WGRAD)
def test_wgrad(fmt, dyadic, blocks, past, M, N):
    announce("bs_gemm_grouped_wgrad", fmt, dyadic, blocks, past, M, N)
    rng = np.random.default_rng(len(blocks) * 10 + M + N)
    b = BLK[fmt]
    sizes = [v * b for v in blocks]
    R = sum(sizes) + past * b
    ac, asc = _operand(rng, M, R, fmt, dyadic)
    bc, bsc = _operand(rng, N, R, fmt, dyadic)
    am, bm = np.float32(2688.0), np.float32(1344.0 if dyadic else 5.0)
    want, _ = OM.grouped_wgrad(_deq(ac, asc, fmt), _deq(bc, bsc, fmt), np.concatenate([[0], np.cumsum(sizes)]))
    nv = fmt == "nvfp4"
    if nv:
        want *= OG.nvfp4_alpha(am, bm)
    ta, tb = torch.tensor([am], device="cuda"), torch.tensor([bm], device="cuda")
    got = bsq.bs_gemm_grouped_wgrad(fmt, *_dev(ac, asc, bc, bsc), _offsets(sizes), ta if nv else None, tb if nv else None)
    assert got.shape == (len(blocks), M, N)
    for e in range(len(blocks)):
        _judge(got[e], want[e], dyadic, (fmt, blocks, M, N, e))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("sizes,N,K", [((2, 1, 3), 100, 160), ((40, 30, 50), 260, 512), ((300, 200, 520), 520, 1024)])
def test_rows_of_a_group_do_not_see_its_neighbours_nan(fmt, sizes, N, K):
    """NaN scales in one group's rows, or in one expert's weights, stay there."""
    announce("bs_gemm_grouped, NaN in one group", fmt, sizes, N, K)
    rng = np.random.default_rng(22)
    E, R = len(sizes), sum(sizes) + 5
    o = np.concatenate([[0], np.cumsum(sizes)])
    a, b = _operand(rng, R, K, fmt, False), _operand(rng, E * N, K, fmt, False)
    am = torch.tensor([3.0], device="cuda") if fmt == "nvfp4" else None
    run = lambda a, b: bsq.bs_gemm_grouped(fmt, *_dev(*a), *(t.view(E, N, -1) for t in _dev(*b)), _offsets(sizes), am, am)
    want = run(a, b)
    assert torch.isfinite(want).all()
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    for bad in range(E):
        for which in (0, 1):
            ops = [list(a), list(b)]
            ops[which][1] = ops[which][1].copy()
            rows = slice(o[bad], o[bad + 1]) if which == 0 else slice(bad * N, bad * N + N)
            ops[which][1][rows] = nan
            got = run(*ops)
            keep = torch.ones(R, dtype=torch.bool, device="cuda")
            keep[o[bad]:o[bad + 1]] = False
            assert torch.equal(got[keep], want[keep]) and torch.isnan(got[~keep]).all(), (bad, which)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("blocks,M,N", [((3, 4, 2), 40, 30), ((5, 9, 30), 128, 200), ((41, 3, 70), 300, 257),
                                        ((60, 10, 60), 1024, 1500)])
def test_wgrad_of_a_group_does_not_see_its_neighbours_nan(fmt, blocks, M, N):
    """NaN scales (and codes, where the format has them) in one group's rows, of
    either operand or both, leave the other groups' products as they are."""
    announce("bs_gemm_grouped_wgrad, NaN in one group", fmt, blocks, M, N)
    rng = np.random.default_rng(21)
    B = BLK[fmt]
    K = sum(blocks) * B
    K = -(-K // 512) * 512                       # aligned rows: the 256 x 256 kernels take them too
    off = _offsets([b * B for b in blocks])
    o = off.cpu().numpy()
    a, b = _operand(rng, M, K, fmt, False), _operand(rng, N, K, fmt, False)
    am = torch.tensor([3.0], device="cuda") if fmt == "nvfp4" else None
    want = bsq.bs_gemm_grouped_wgrad(fmt, *_dev(*a), *_dev(*b), off, am, am)
    assert torch.isfinite(want).all()
    per = 1 if fmt == "mxfp8" else 2
    nan_scale = 0x7F if fmt == "nvfp4" else 0xFF
    for bad in range(-1, len(blocks)):           # -1: the rows past the last group
        k0, k1 = (o[bad], o[bad + 1]) if bad >= 0 else (o[-1], K)
        for which in (1, 2, 3):
            ops = []
            for i, (codes, scales) in enumerate((a, b)):
                codes, scales = codes.copy(), scales.copy()
                if which >> i & 1:
                    scales[:, k0 // B:k1 // B] = nan_scale
                    if fmt == "mxfp8":
                        codes[:, k0 // per:k1 // per] = 0x7F
                ops += _dev(codes, scales)
            got = bsq.bs_gemm_grouped_wgrad(fmt, *ops, off, am, am)
            for e in range(len(blocks)):
                if e != bad:
                    assert torch.equal(got[e], want[e]), (bad, which, e)


def test_wgrad_offsets_inside_a_block_are_rounded_down():
    announce("bs_gemm_grouped_wgrad unaligned offsets")
    rng = np.random.default_rng(3)
    ops = _dev(*_operand(rng, 20, 128, "mxfp4", True), *_operand(rng, 24, 128, "mxfp4", True))
    f = lambda o: bsq.bs_gemm_grouped_wgrad("mxfp4", *ops, torch.tensor(o, dtype=torch.int32, device="cuda"))
    assert torch.equal(f([5, 63, 127]), f([0, 32, 96]))


def test_graph_and_other_stream():
    announce("grouped products in a graph")
    rng = np.random.default_rng(4)
    a, b = _dev(*_operand(rng, 96, 256, "nvfp4", False)), _dev(*_operand(rng, 3 * 64, 256, "nvfp4", False))
    b = tuple(v.view(3, 64, -1) for v in b)
    wa, wb = _dev(*_operand(rng, 64, 96, "mxfp8", False)), _dev(*_operand(rng, 32, 96, "mxfp8", False))
    off, am = _offsets([32, 0, 64]), torch.tensor([3.0], device="cuda")

    def call():
        return (bsq.bs_gemm_grouped("nvfp4", *a, *b, off, am, am), bsq.bs_gemm_grouped_wgrad("mxfp8", *wa, *wb, off))
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = call()
    for n in range(3):
        for t in rec:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(want, got, rec)), n
        call()


def test_refusals():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    off = _offsets([1, 3])
    with pytest.raises(ValueError):
        bsq.bs_gemm_grouped("fp8", z(4, 32), z(4, 1), z(2, 8, 32), z(2, 8, 1), off)
    with pytest.raises(ValueError):
        bsq.bs_gemm_grouped("nvfp4", z(4, 16), z(4, 2), z(2, 8, 16), z(2, 8, 2), off)       # amaxes missing
    with pytest.raises(ValueError):
        bsq.bs_gemm_grouped("mxfp4", z(4, 16), z(4, 1), z(3, 8, 16), z(3, 8, 1), off)       # three experts, two groups
    with pytest.raises(ValueError):
        bsq.bs_gemm_grouped("mxfp4", z(4, 16), z(4, 2), z(2, 8, 16), z(2, 8, 1), off)       # scales
    with pytest.raises(ValueError):
        bsq.bs_gemm_grouped("mxfp4", z(4, 16), z(4, 1), z(2, 8, 16), z(2, 8, 1), off.long())
    with pytest.raises(ValueError):
        bsq.bs_gemm_grouped_wgrad("mxfp4", z(4, 16), z(4, 1), z(2, 32), z(2, 2), off)       # other rows
