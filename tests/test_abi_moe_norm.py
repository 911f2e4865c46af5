"""Refusals of the norm, router and grouped-product entry points (no GPU: argument
errors return before any HIP call)."""

import ctypes
import os

import pytest

import fp8_quantized_gemm_amd as bsq
from oracle import moe as OM

pytestmark = pytest.mark.skipif(not os.path.exists(bsq.LIB_PATH),
                                reason="libbsq.so not built (run __graft_entry__.build())")

A = 0x1000000          # 16-byte aligned addresses far apart, never dereferenced
B, C, D, E_, F, G = (A + i * 0x1000000 for i in range(1, 7))
EINVAL, EUNSUP, OK = bsq.BSQ_EINVAL, bsq.BSQ_EUNSUPPORTED, bsq.BSQ_OK


def _norm(**kw):
    a = dict(x=A, t=0, o=B, rows=8, cols=64, wq=C, kind=0, gate=None, alpha=1.0, wp=C, eps=1e-6, r=D, h=E_, rq=F, rp=F,
             amax=G)
    a.update(kw)
    return bsq.lib().block_norm(a["x"], a["t"], a["o"], a["rows"], a["cols"], a["wq"], a["kind"], a["gate"], a["alpha"],
                                a["wp"], a["eps"], a["r"], a["h"], a["rq"], a["rp"], a["amax"], None)


def test_block_norm_refusals():
    assert _norm(rows=-1) == EINVAL and _norm(cols=0) == EINVAL
    assert _norm(cols=16385) == EUNSUP
    assert _norm(t=2) == EINVAL and _norm(kind=4) == EINVAL
    assert _norm(eps=0.0) == EINVAL and _norm(eps=float("nan")) == EINVAL
    assert _norm(o=None) == EINVAL                           # w_post without o
    assert _norm(o=None, wq=None, rq=None) == EINVAL         # r without o
    assert _norm(o=None, wq=None, rq=None, r=None, wp=None, h=None, rp=None, amax=None) == EINVAL
    assert _norm(r=None) == EINVAL and _norm(h=None) == EINVAL
    assert _norm(wp=None) == EINVAL                          # h without w_pre
    assert _norm(kind=1) == EINVAL and _norm(gate=C) == EINVAL
    assert _norm(wq=None) == EINVAL                          # rstd_post without w_post
    assert _norm(x=None) == EINVAL and _norm(x=A + 1) == EINVAL and _norm(wp=C + 2) == EINVAL
    assert _norm(r=A) == EINVAL and _norm(h=B + 64) == EINVAL and _norm(h=D) == EINVAL   # overlaps
    assert _norm(rows=1 << 40, cols=16384) == EINVAL
    assert _norm(rows=0, amax=None) == OK


def _norm_bwd(**kw):
    a = dict(r=A, t=0, o=B, dr=C, dh=D, rows=8, cols=64, wq=E_, kind=0, gate=None, alpha=1.0, wp=E_, rq=F, rp=F, dx=G,
             do=G + 0x10000, dg=None, dwp=G + 0x20000, dwq=G + 0x30000, ws=G + 0x40000, wsb=1 << 20)
    a.update(kw)
    return bsq.lib().block_norm_backward(a["r"], a["t"], a["o"], a["dr"], a["dh"], a["rows"], a["cols"], a["wq"],
                                         a["kind"], a["gate"], a["alpha"], a["wp"], a["rq"], a["rp"], a["dx"], a["do"],
                                         a["dg"], a["dwp"], a["dwq"], a["ws"], a["wsb"], None)


def test_block_norm_backward_refusals():
    need = ctypes.c_int64(0)
    assert bsq.lib().block_norm_backward_workspace(8, 64, ctypes.byref(need)) == OK and need.value > 0
    assert bsq.lib().block_norm_backward_workspace(8, 64, None) == EINVAL
    assert _norm_bwd(wsb=need.value - 1) == EINVAL and _norm_bwd(ws=None) == EINVAL and _norm_bwd(ws=G + 4) == EINVAL
    assert _norm_bwd(dx=None) == EINVAL and _norm_bwd(do=None) == EINVAL
    assert _norm_bwd(dh=None) == EINVAL and _norm_bwd(rp=None) == EINVAL and _norm_bwd(rq=None) == EINVAL
    assert _norm_bwd(dwp=None) == EINVAL and _norm_bwd(dwq=None) == EINVAL
    assert _norm_bwd(kind=1, gate=F) == EINVAL               # no d_gate
    assert _norm_bwd(wp=None, dwp=None, dh=None, rp=None, dr=None) == EINVAL   # no incoming gradient
    assert _norm_bwd(dx=A) == EINVAL and _norm_bwd(do=G) == EINVAL             # overlaps
    assert _norm_bwd(cols=20000) == EUNSUP


def test_moe_rows():
    for T, E, k, al in ((0, 8, 2, 32), (1, 8, 2, 1), (1, 8, 2, 16), (100, 64, 6, 32), (4096, 8, 2, 128), (3, 512, 16, 512)):
        assert bsq.moe_rows(T, E, k, al) == OM.rows_bound(T, E, k, al)
    n = ctypes.c_int64(0)
    L = bsq.lib()
    assert L.moe_rows(4, 8, 2, 1, None) == EINVAL
    assert L.moe_rows(4, 8, 9, 1, ctypes.byref(n)) == EINVAL          # k > experts
    assert L.moe_rows(4, 513, 2, 1, ctypes.byref(n)) == EUNSUP
    assert L.moe_rows(4, 64, 17, 1, ctypes.byref(n)) == EUNSUP
    assert L.moe_rows(4, 8, 2, 0, ctypes.byref(n)) == EINVAL and L.moe_rows(4, 8, 2, 513, ctypes.byref(n)) == EINVAL
    assert L.moe_rows(1 << 30, 8, 2, 1, ctypes.byref(n)) == EINVAL    # 2^31 assignments
    assert L.moe_rows(-1, 8, 2, 1, ctypes.byref(n)) == EINVAL


def _route(**kw):
    a = dict(lg=A, t=0, T=16, E=8, k=2, bias=None, sc=0, al=1, rows=32, ids=B, w=C, off=D, ro=E_, src=F, ws=G, wsb=1 << 20)
    a.update(kw)
    return bsq.lib().moe_route(a["lg"], a["t"], a["T"], a["E"], a["k"], a["bias"], a["sc"], 1, 1.0, a["al"], a["rows"],
                               a["ids"], a["w"], a["off"], a["ro"], a["src"], a["ws"], a["wsb"], None)


def test_moe_route_refusals():
    assert _route(rows=31) == EINVAL and _route(al=16) == EINVAL       # src shorter than the bound
    assert _route(k=0) == EINVAL and _route(k=9) == EINVAL and _route(E=600) == EUNSUP
    assert _route(sc=2) == EINVAL and _route(t=3) == EINVAL
    for p in ("lg", "ids", "w", "off", "ro", "src"):
        assert _route(**{p: None}) == EINVAL, p
    assert _route(ids=B + 2) == EINVAL and _route(lg=A + 1) == EINVAL and _route(bias=A + 2) == EINVAL
    assert _route(T=128, rows=256, ws=None) == EINVAL and _route(T=128, rows=256, wsb=4) == EINVAL
    L = bsq.lib()
    assert L.moe_route_backward(A, 0, 16, 8, 2, B, C, 0, 1, 1.0, A, None) == EINVAL    # overlap
    assert L.moe_route_backward(A, 0, 16, 8, 2, None, C, 0, 1, 1.0, D, None) == EINVAL
    assert L.moe_route_backward(A, 0, 0, 8, 2, None, None, 0, 1, 1.0, None, None) == OK


def test_mover_refusals():
    L = bsq.lib()
    assert L.moe_gather(A, 4, 64, 0, B, 8, C, None) == EINVAL
    assert L.moe_gather(A, 4, 64, 2, None, 8, C, None) == EINVAL
    assert L.moe_gather(A, 4, 64, 2, B, 8, A, None) == EINVAL          # overlap
    assert L.moe_gather(A, 4, 64, 2, B, 0, C, None) == OK
    assert L.moe_gather(A, 4, 64, 2, B, 1 << 31, C, None) == EINVAL
    assert L.moe_combine(A, 8, 64, None, None, 4, 2, C, None) == EINVAL
    assert L.moe_combine(A, 8, 64, B, None, 4, 2, A + 16, None) == EINVAL
    assert L.moe_combine(A, 8, 64, B, None, 0, 2, None, None) == OK
    assert L.moe_combine_backward(A, B, 4, 64, 2, C, D, None, 8, E_, F, None) == EINVAL
    assert L.moe_combine_backward(A, B, 4, 64, 2, C, D, G, 8, B, F, None) == EINVAL    # d_y over y
    assert L.moe_combine_backward(A, B, 4, 64, 2, None, D, G, 8, E_, F, None) == EINVAL
    wide = (1 << 30) + 1
    assert L.moe_gather(A, 1, wide, 2, B, 0, C, None) == EUNSUP
    assert L.moe_combine(A, 0, wide, B, None, 1, 2, C, None) == EUNSUP
    assert L.moe_combine_backward(A, B, 1, wide, 2, C, D, G, 0, E_, F, None) == EUNSUP


def _grouped(**kw):
    a = dict(fmt=0, E=4, off=A, rows=32, N=64, K=64, ac=B, as_=B, aa=C, bc=D, bs=D, ba=C, bn=4, c=E_, ldc=64)
    a.update(kw)
    return bsq.lib().bs_gemm_grouped(a["fmt"], a["E"], a["off"], a["rows"], a["N"], a["K"], a["ac"], a["as_"], a["aa"],
                                     a["bc"], a["bs"], a["ba"], a["bn"], a["c"], a["ldc"], None)


def test_bs_gemm_grouped_refusals():
    assert _grouped(fmt=3) == EUNSUP and _grouped(fmt=9) == EINVAL
    assert _grouped(E=0) == EINVAL and _grouped(E=4097) == EINVAL
    assert _grouped(K=40) == EINVAL and _grouped(fmt=1, K=48) == EINVAL and _grouped(ldc=63) == EINVAL
    assert _grouped(off=None) == EINVAL and _grouped(c=None) == EINVAL and _grouped(ac=None) == EINVAL
    assert _grouped(aa=None) == EINVAL and _grouped(ba=None) == EINVAL and _grouped(bn=3) == EINVAL
    assert _grouped(ac=B + 8) == EINVAL and _grouped(c=E_ + 1) == EINVAL and _grouped(off=A + 2) == EINVAL
    assert _grouped(rows=1 << 31) == EINVAL and _grouped(N=1 << 40, ldc=1 << 40) == EINVAL
    assert _grouped(rows=0) == OK and _grouped(N=0, ldc=0) == OK


def test_bs_gemm_grouped_wgrad_refusals():
    def f(fmt=0, E=4, off=A, M=64, N=64, rows=32, ac=B, aa=C, bc=D, c=E_):
        return bsq.lib().bs_gemm_grouped_wgrad(fmt, E, off, M, N, rows, ac, B, aa, bc, D, C, c, None)
    assert f(fmt=3) == EUNSUP and f(E=0) == EINVAL and f(rows=24) == EINVAL and f(fmt=2, rows=48) == EINVAL
    assert f(off=None) == EINVAL and f(c=None) == EINVAL and f(ac=None) == EINVAL and f(aa=None) == EINVAL
    assert f(bc=D + 4) == EINVAL and f(M=-1) == EINVAL and f(M=0) == OK
