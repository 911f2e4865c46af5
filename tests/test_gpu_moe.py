"""Router, gather, combine and their gradients against the oracle: integers exact;
FP32 weights within 32 roundings (exp, log1p and the division are a few units, the
sums have at most 9 + 6 steps); BF16 rows half a step plus the FP32 sum."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from oracle import moe as OM

from _gpu import announce, gpu

pytestmark = gpu

U = 2.0 ** -24


def _logits(T, E, dtype, seed, ties=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = 3 * torch.randn((T, E), generator=g, device="cuda")
    if ties:
        l = torch.round(l)                               # many equal scores
    if T > 4:
        l[torch.rand((T, E), generator=g, device="cuda") < 0.1] = float("-inf")
        l[1] = float("-inf")                             # a token without any expert
        l[2, 1:] = float("-inf")                         # ... with one
        l[3] = torch.finfo(torch.float32).min if dtype == torch.float32 else torch.finfo(torch.bfloat16).min
        l[4, 0] = float("nan")                           # masked
    return l.to(dtype)


ROUTES = [  # tokens, experts, k, align, bias, dtype, ties
    (1, 8, 2, 1, False, torch.float32, False),
    (1, 1, 1, 1, False, torch.bfloat16, False),
    (7, 5, 5, 1, True, torch.float32, True),
    (16, 64, 4, 1, True, torch.bfloat16, True),
    (63, 60, 6, 16, False, torch.float32, True),
    (64, 512, 16, 32, True, torch.float32, False),
    (65, 128, 8, 32, True, torch.bfloat16, True),
    (500, 160, 6, 16, False, torch.float32, False),
    (1000, 8, 2, 32, True, torch.bfloat16, True),
    (2051, 300, 3, 128, False, torch.float32, True),
    (9000, 16, 1, 1, True, torch.float32, False),
]


@pytest.mark.parametrize("T,E,k,align,bias,dtype,ties", ROUTES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route(T, E, k, align, bias, dtype, ties, scoring, normalize):
    announce("moe_route", T, E, k, align, bias, dtype, ties, scoring, normalize)
    l = _logits(T, E, dtype, T + E, ties)
    b = torch.round(4 * torch.randn(E, device="cuda")) / 4 if bias else None
    f = bsq.moe_route(l, k, b, scoring, normalize, 1.5, align)
    ln, bn = l.float().cpu().numpy(), None if b is None else b.cpu().numpy()
    w = OM.route(ln, k, bn, scoring, normalize, 1.5, align)
    for name in ("experts", "offsets", "row_of", "src"):
        assert np.array_equal(f[name].cpu().numpy(), w[name]), name
    got = f["weights"].double().cpu().numpy()
    # exp(l - max): the difference is exact to half a unit of |l| + |max| <= 30, a relative
    # error of 30 U in the power; for -inf .. lowest values the weights are 0 or equal
    assert np.all(np.abs(got - w["weights"]) <= 64 * U * np.abs(w["weights"]) + 1e-37)
    d = torch.randn((T, k), device="cuda")
    g = bsq.moe_route_backward(l, f["experts"], d, scoring, normalize, 1.5)
    assert g.dtype == dtype
    want = OM.route_backward(ln, w["experts"], d.double().cpu().numpy(), scoring, normalize, 1.5)
    mag = np.zeros((T, E))                               # terms of a logit's gradient
    dm = np.abs(d.double().cpu().numpy()) * 1.5
    rowmax = dm.max(1, initial=0)[:, None]
    mag += rowmax * (np.abs(want) > 0)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    tol = 128 * U * mag + half * np.abs(want) + 1e-37
    assert np.all(np.abs(g.double().cpu().numpy() - want) <= tol)


def test_route_no_tokens_and_all_masked():
    announce("moe_route without tokens, with every logit masked")
    f = bsq.moe_route(torch.zeros((0, 8), device="cuda"), 2, align=16)
    assert f["src"].numel() == 0 and f["offsets"].tolist() == [0] * 9
    f = bsq.moe_route(torch.full((70, 8), float("-inf"), device="cuda"), 2, align=16)
    assert torch.all(f["experts"] == -1) and torch.all(f["src"] == -1) and not f["weights"].any()
    assert not f["offsets"].any()
    g = bsq.moe_route_backward(torch.full((70, 8), float("-inf"), device="cuda"), f["experts"],
                               torch.ones((70, 2), device="cuda"), normalize=False)
    assert not g.any()


def test_route_one_expert_takes_all():
    announce("moe_route to one expert")
    l = torch.zeros((777, 64), device="cuda")
    l[:, 63] = 5
    f = bsq.moe_route(l, 1, align=32)
    assert torch.all(f["experts"] == 63) and f["offsets"][63].item() == 0 and f["offsets"][64].item() == 800
    assert torch.equal(f["row_of"].flatten(), torch.arange(777, device="cuda", dtype=torch.int32))


MOVES = [(1, 8, 2, 1, 64), (5, 3, 2, 16, 7), (33, 16, 4, 1, 2048), (100, 8, 2, 32, 1408), (300, 64, 6, 16, 520), (129, 4, 1, 1, 1001)]


@pytest.mark.parametrize("T,E,k,align,C", MOVES)
def test_gather_and_combine(T, E, k, align, C):
    announce("moe_gather / moe_combine", T, E, k, align, C)
    g = torch.Generator(device="cuda").manual_seed(T * 7 + C)
    f = bsq.moe_route(_logits(T, E, torch.float32, T), k, align=align)
    src, row_of = f["src"].cpu().numpy(), f["row_of"].cpu().numpy()
    x = torch.randn((T, C), generator=g, device="cuda").bfloat16()
    xp = bsq.moe_gather(x, f["src"], k)
    assert np.array_equal(xp.double().cpu().numpy(), OM.gather(x.double().cpu().numpy(), src, k))
    y = torch.randn((len(src), C), generator=g, device="cuda").bfloat16()
    yn = y.double().cpu().numpy()
    for w in (None, f["weights"]):
        got = bsq.moe_combine(y, f["row_of"], w).double().cpu().numpy()
        wn = None if w is None else w.double().cpu().numpy()
        want = OM.combine(yn, row_of, wn)
        mag = OM.combine(np.abs(yn), row_of, wn)         # weights are not negative
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2 * k + 2) * U * mag)
    d = torch.randn((T, C), generator=g, device="cuda").bfloat16()
    dy, dw = bsq.moe_combine_backward(d, y, f["src"], f["row_of"], f["weights"])
    wy, ww = OM.combine_backward(d.double().cpu().numpy(), yn, src, row_of, f["weights"].double().cpu().numpy())
    _, mw = OM.combine_backward(np.abs(d.double().cpu().numpy()), np.abs(yn), src, row_of, np.ones((T, k)))
    assert np.all(np.abs(dy.double().cpu().numpy() - wy) <= 2.0 ** -8 * np.abs(wy) + 2 * U * np.abs(wy))
    # products exact in FP32 (16 significant bits); at most C / 64 + 6 additions in one chain
    assert np.all(np.abs(dw.double().cpu().numpy() - ww) <= (C / 64 + 16) * U * mw)


@pytest.mark.parametrize("C", [64, 1000, 1001])
def test_rows_at_any_element_alignment(C):
    """The same rows, one element off 16-byte alignment, give the same bits."""
    announce("movers, unaligned", C)
    off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)
    f = bsq.moe_route(_logits(57, 16, torch.float32, C), 3, align=16)
    x, y, d = (torch.randn((n, C), device="cuda").bfloat16() for n in (57, len(f["src"]), 57))
    assert torch.equal(bsq.moe_gather(off(x), f["src"], 3), bsq.moe_gather(x, f["src"], 3))
    for w in (None, f["weights"]):
        assert torch.equal(bsq.moe_combine(off(y), f["row_of"], w), bsq.moe_combine(y, f["row_of"], w))
    got = bsq.moe_combine_backward(off(d), off(y), f["src"], f["row_of"], f["weights"])
    want = bsq.moe_combine_backward(d, y, f["src"], f["row_of"], f["weights"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,k,C", [(7001, 2, 2048), (1700, 3, 8192), (900, 2, 16384 + 64), (515, 4, 1088), (65, 8, 320)])
def test_gather_in_column_slabs(T, k, C):
    """Every column is moved once, however the columns are divided."""
    announce("moe_gather, many columns", T, k, C)
    f = bsq.moe_route(_logits(T, 8, torch.float32, C), k, align=16)
    x = torch.randn((T, C), device="cuda").bfloat16()
    out = torch.full((len(f["src"]), C), 7.0, device="cuda").bfloat16()
    bsq.moe_gather(x, f["src"], k, out=out)
    src = f["src"].long()
    want = x[src.clamp(min=0) // k]
    want[src < 0] = 0
    assert torch.equal(out, want)


def test_rows_past_32_bit_offsets():
    """2^20 + 8 rows of 4,096: elements past 2^32."""
    announce("movers, rows past 2^32 elements")
    T, k, C, rows = 8, 2, 4096, (1 << 20) + 8
    x = torch.randn((T, C), device="cuda").bfloat16()
    src = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    place = torch.tensor([0, 1, 1 << 18, (1 << 19) - 1, 1 << 19, (1 << 19) + 3, 5, 6, 7, 8, 9, 10, 11,
                          1 << 20, (1 << 20) + 1, rows - 1], dtype=torch.int32, device="cuda")
    src[place.long()] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    xp = bsq.moe_gather(x, src, k)
    assert torch.equal(xp[place.long()], x.repeat_interleave(k, 0))
    assert int(torch.count_nonzero(xp[12:1 << 18])) == 0 and int(torch.count_nonzero(xp[(1 << 20) + 2:rows - 1])) == 0
    row_of, w = place.view(T, k), torch.rand((T, k), device="cuda")
    small = torch.arange(T * k, dtype=torch.int32, device="cuda")
    y = xp[place.long()]
    assert torch.equal(bsq.moe_combine(xp, row_of, w), bsq.moe_combine(y, small.view(T, k), w))
    want = bsq.moe_combine_backward(x, y, small, small.view(T, k), w)
    del y
    got = bsq.moe_combine_backward(x, xp, src, row_of, w)
    assert torch.equal(got[0][place.long()], want[0]) and torch.equal(got[1], want[1])


def test_indices_out_of_range_are_no_assignment():
    announce("gather / combine with out-of-range indices")
    x = torch.randn((4, 64), device="cuda").bfloat16()
    src = torch.tensor([0, 7, 8, 1 << 30, -5, 3], dtype=torch.int32, device="cuda")
    out = bsq.moe_gather(x, src, 2)
    assert torch.equal(out[0], x[0]) and torch.equal(out[1], x[3]) and torch.equal(out[5], x[1])
    assert not out[2:5].any()
    ro = torch.tensor([[0, 4], [6, -1]], dtype=torch.int32, device="cuda")
    y = torch.randn((5, 64), device="cuda").bfloat16()
    c = bsq.moe_combine(y, ro)
    assert torch.equal(c[0], (y[0].float() + y[4].float()).bfloat16()) and not c[1].any()


def test_other_stream_and_graph():
    announce("moe_route and movers in a graph")
    l = _logits(700, 32, torch.float32, 3)
    x = torch.randn((700, 256), device="cuda").bfloat16()

    def call():
        f = bsq.moe_route(l, 4, align=16)
        xp = bsq.moe_gather(x, f["src"], 4)
        out = bsq.moe_combine(xp, f["row_of"], f["weights"])
        dy, dw = bsq.moe_combine_backward(x, xp, f["src"], f["row_of"], f["weights"])
        g = bsq.moe_route_backward(l, f["experts"], dw)
        return dict(f, xp=xp, out=out, dy=dy, dw=dw, g=g)
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
        for t in rec.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(v, got[k]) and torch.equal(v, rec[k]), (n, k)
        call()


def test_refusals():
    l = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        bsq.moe_route(l, 2, scoring="other")
    with pytest.raises(ValueError):
        bsq.moe_route(l, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(bsq.BsqError):
        bsq.moe_route(l, 9)
    with pytest.raises(ValueError):
        bsq.moe_gather(l.bfloat16(), torch.zeros(4, device="cuda"), 2)
    with pytest.raises(ValueError):
        bsq.moe_combine(l.bfloat16(), torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 1), device="cuda"))
