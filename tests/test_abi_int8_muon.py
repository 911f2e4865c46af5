"""Refusals of the 8-bit integer and the orthogonalised-update entry points (no GPU:
argument errors return before any HIP call)."""

import ctypes
import os

import pytest
import torch

import fp8_quantized_gemm_amd as bsq

pytestmark = pytest.mark.skipif(not os.path.exists(bsq.LIB_PATH),
                                reason="libbsq.so not built (run __graft_entry__.build())")

A = 0x1000000          # 256-byte aligned addresses far apart, never dereferenced
B, C, D, E_, F, G = (A + i * 0x1000000 for i in range(1, 7))
EINVAL, EUNSUP, OK = bsq.BSQ_EINVAL, bsq.BSQ_EUNSUPPORTED, bsq.BSQ_OK


def _q(x=A, rows=8, cols=64, codes=B, scales=C):
    return bsq.lib().int8_quantize(x, rows, cols, codes, scales, None)


def test_int8_quantize_refusals():
    assert _q(rows=-1) == EINVAL and _q(cols=-1) == EINVAL and _q(rows=1 << 40, cols=1 << 20) == EINVAL
    assert _q(x=None) == EINVAL and _q(codes=None) == EINVAL and _q(scales=None) == EINVAL
    assert _q(x=A + 2) == EINVAL and _q(codes=B + 8) == EINVAL and _q(scales=C + 2) == EINVAL
    assert _q(codes=A) == EINVAL and _q(scales=A + 64) == EINVAL and _q(scales=B) == EINVAL      # overlaps
    assert _q(rows=0) == OK and _q(rows=0, x=None, codes=None, scales=None) == OK


def _qt(**kw):
    a = dict(x=A, rows=8, cols=64, rc=B, rs=C, cc=D, cs=E_, ws=F, wsb=(8 + 64) * 4)
    a.update(kw)
    return bsq.lib().int8_quantize_transpose(a["x"], a["rows"], a["cols"], a["rc"], a["rs"], a["cc"], a["cs"], a["ws"],
                                             a["wsb"], None)


def test_int8_quantize_transpose_refusals():
    n = ctypes.c_int64(0)
    L = bsq.lib()
    assert L.int8_quantize_transpose_workspace(8, 64, ctypes.byref(n)) == OK and n.value == 288
    assert L.int8_quantize_transpose_workspace(8, 64, None) == EINVAL
    assert L.int8_quantize_transpose_workspace(-1, 64, ctypes.byref(n)) == EINVAL
    assert _qt(x=None) == EINVAL and _qt(rs=None) == EINVAL and _qt(rc=None) == EINVAL and _qt(cs=None) == EINVAL
    assert _qt(rc=None, rs=None, cc=None, cs=None) == EINVAL
    assert _qt(ws=None) == EINVAL and _qt(wsb=287) == EINVAL and _qt(ws=F + 2) == EINVAL
    assert _qt(x=A + 8) == EINVAL and _qt(rc=B + 4) == EINVAL and _qt(cc=D + 4) == EINVAL and _qt(cs=E_ + 1) == EINVAL
    assert _qt(cc=B) == EINVAL and _qt(ws=A) == EINVAL and _qt(cs=C) == EINVAL                   # overlaps
    assert _qt(rows=-1) == EINVAL and _qt(rows=1 << 40, cols=1 << 20) == EINVAL
    assert _qt(rows=0, cols=0) == OK


def _g(**kw):
    a = dict(M=8, N=32, K=64, a=A, sa=B, b=C, sb=D, bias=None, c=E_, ldc=32)
    a.update(kw)
    return bsq.lib().int8_gemm(a["M"], a["N"], a["K"], a["a"], a["sa"], a["b"], a["sb"], a["bias"], a["c"], a["ldc"], None)


def _l(**kw):
    a = dict(x=A, M=8, N=32, K=64, w=C, sw=D, bias=None, c=E_, ldc=32, ws=F, wsb=1 << 20)
    a.update(kw)
    return bsq.lib().int8_linear(a["x"], a["M"], a["N"], a["K"], a["w"], a["sw"], a["bias"], a["c"], a["ldc"], a["ws"],
                                 a["wsb"], None)


def test_int8_product_refusals():
    for f in (_g, _l):
        assert f(M=-1) == EINVAL and f(N=-1) == EINVAL and f(K=-1) == EINVAL and f(ldc=31) == EINVAL
        assert f(K=1 << 17) == EUNSUP
        assert f(M=1 << 40, K=1 << 16) == EINVAL and f(M=1 << 35) == EINVAL
        assert f(c=None) == EINVAL and f(c=E_ + 1) == EINVAL and f(bias=G + 2) == EINVAL
        assert f(M=0) == OK and f(N=0, ldc=0) == OK
    assert _g(a=None) == EINVAL and _g(b=None) == EINVAL and _g(sa=None) == EINVAL and _g(sb=None) == EINVAL
    assert _g(a=A + 8) == EINVAL and _g(b=C + 8) == EINVAL and _g(sa=B + 2) == EINVAL and _g(sb=D + 2) == EINVAL
    assert _g(c=A) == EINVAL and _g(c=C) == EINVAL and _g(c=B) == EINVAL and _g(c=D) == EINVAL and _g(bias=E_) == EINVAL
    assert _l(x=None) == EINVAL and _l(w=None) == EINVAL and _l(sw=None) == EINVAL and _l(x=A + 8) == EINVAL
    assert _l(ws=None) == EINVAL and _l(ws=F + 8) == EINVAL
    assert _l(ws=A) == EINVAL and _l(ws=C) == EINVAL and _l(ws=E_) == EINVAL and _l(c=A) == EINVAL
    n = ctypes.c_int64(0)
    assert bsq.lib().int8_linear_workspace(8, 64, ctypes.byref(n)) == OK and n.value >= 8 * 64 + 32
    assert _l(wsb=n.value - 1) == EINVAL
    assert bsq.lib().int8_linear_workspace(8, 64, None) == EINVAL
    assert bsq.lib().int8_linear_workspace(-8, 64, ctypes.byref(n)) == EINVAL


COEFS = (ctypes.c_float * 15)(*([3.4445, -4.7750, 2.0315] * 5))


def _o(**kw):
    a = dict(x=A, t=0, batch=2, rows=8, cols=64, steps=5, coefs=COEFS, eps=1e-7, out=B, ws=C, wsb=1 << 24)
    a.update(kw)
    return bsq.lib().orthogonalize(a["x"], a["t"], a["batch"], a["rows"], a["cols"], a["steps"], a["coefs"], a["eps"],
                                   a["out"], a["ws"], a["wsb"], None)


def test_orthogonalize_refusals():
    n = ctypes.c_int64(0)
    L = bsq.lib()
    assert L.orthogonalize_workspace(2, 8, 64, ctypes.byref(n)) == OK and n.value > 0
    assert _o(wsb=n.value - 1) == EINVAL
    assert L.orthogonalize_workspace(2, 8, 64, None) == EINVAL
    assert L.orthogonalize_workspace(2, -8, 64, ctypes.byref(n)) == EINVAL
    assert L.orthogonalize_workspace(1, 1 << 22, 8, ctypes.byref(n)) == EUNSUP
    assert L.orthogonalize_workspace(65536, 8, 8, ctypes.byref(n)) == EUNSUP
    assert L.orthogonalize_workspace(0, 8, 8, ctypes.byref(n)) == OK and n.value == 0
    assert _o(batch=-1) == EINVAL and _o(rows=-1) == EINVAL and _o(cols=1 << 22) == EUNSUP
    assert _o(steps=0) == EINVAL and _o(steps=33) == EINVAL and _o(coefs=None) == EINVAL
    assert _o(eps=0.0) == EINVAL and _o(eps=-1.0) == EINVAL and _o(eps=float("nan")) == EINVAL
    assert _o(t=2) == EINVAL and _o(x=None) == EINVAL and _o(out=None) == EINVAL
    assert _o(x=A + 1) == EINVAL and _o(t=1, x=A + 2) == EINVAL and _o(out=B + 1) == EINVAL
    assert _o(ws=None) == EINVAL and _o(ws=C + 16) == EINVAL
    assert _o(out=A) == EINVAL and _o(ws=A) == EINVAL and _o(ws=B) == EINVAL
    assert _o(rows=0) == OK


def _m(**kw):
    a = dict(w=A, m=B, g=C, batch=2, rows=8, cols=64, steps=5, coefs=COEFS, eps=1e-7, wb=D, amax=None, ws=E_, wsb=1 << 24)
    a.update(kw)
    return bsq.lib().muon_update(a["w"], a["m"], a["g"], a["batch"], a["rows"], a["cols"], 1e-3, 0.95, 1, 0.0, 1.0,
                                 a["steps"], a["coefs"], a["eps"], a["wb"], a["amax"], a["ws"], a["wsb"], None)


def test_muon_update_refusals():
    for k in ("w", "m", "g", "wb", "ws"):
        assert _m(**{k: None}) == EINVAL, k
    assert _m(w=A + 2) == EINVAL and _m(m=B + 2) == EINVAL and _m(g=C + 1) == EINVAL and _m(wb=D + 1) == EINVAL
    assert _m(amax=F + 2) == EINVAL and _m(ws=E_ + 16) == EINVAL and _m(wsb=64) == EINVAL
    assert _m(m=A) == EINVAL and _m(g=A) == EINVAL and _m(wb=B) == EINVAL and _m(amax=A) == EINVAL and _m(ws=D) == EINVAL
    assert _m(steps=0) == EINVAL and _m(coefs=None) == EINVAL and _m(eps=0.0) == EINVAL and _m(rows=1 << 22) == EUNSUP
    assert _m(batch=0) == OK


def test_python_refusals():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)             # not on a GPU
    w, s = torch.zeros(8, 16, dtype=torch.int8), torch.ones(8)
    for call in (lambda: bsq.int8_quantize(x), lambda: bsq.int8_quantize_transpose(x), lambda: bsq.int8_linear(x, w, s),
                 lambda: bsq.orthogonalize(x), lambda: bsq.int8_gemm(w, s, w, s),
                 lambda: bsq.int8_gemm(w.view(torch.uint8), s, w, s), lambda: bsq.int8_gemm(w, s[:4], w, s),
                 lambda: bsq.int8_gemm(w, s, w[:, :8], s), lambda: bsq.int8_gemm(w, s, w, s, bias=s[:3]),
                 lambda: bsq.muon_update(torch.zeros(4, 16), torch.zeros(4, 16), x, 1e-3)):
        with pytest.raises(ValueError):
            call()


def test_coefficient_checks():
    assert list(bsq._coefs(2, (1.0, 2.0, 3.0))) == [1, 2, 3, 1, 2, 3]
    assert list(bsq._coefs(2, bsq._coef_key([[1, 2, 3], (4, 5, 6)]))) == [1, 2, 3, 4, 5, 6]
    for steps, c in ((0, (1, 2, 3)), (2, (1, 2)), (2, ((1, 2, 3),)), (1, ()), (1, ("a", 1, 2)), (3, ((1, 2, 3), (1, 2, 3)))):
        with pytest.raises(ValueError):
            bsq._coefs(steps, bsq._coef_key(c))
