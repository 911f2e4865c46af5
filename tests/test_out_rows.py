"""Outputs whose rows overlap (expanded or strided tensors) are refused: with a row stride
of N in their place the library would write past them."""

import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from _gpu import gpu


def test_row_stride():
    buf = torch.empty(4, 24)
    assert bsq._row_stride(buf) == 24 and bsq._row_stride(buf[:, :8]) == 24 and bsq._row_stride(buf[:, :1]) == 24
    assert bsq._row_stride(buf[:1].expand(4, 24)) == 0                          # the library refuses ldc < N
    assert bsq._row_stride(buf.view(-1).as_strided((4, 24), (23, 1))) == 23
    assert bsq._row_stride(buf[:1, :8]) == 8 and bsq._row_stride(torch.empty(96).as_strided((1, 8), (1, 1))) == 8
    assert bsq._row_stride(torch.empty(0, 8)) == 8


def _calls():
    z8 = lambda *s: torch.zeros(s, dtype=torch.int8, device="cuda")
    one = lambda n: torch.ones(n, device="cuda")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    yield lambda out: bsq.int8_gemm(z8(4, 64), one(4), z8(24, 64), one(24), out=out)
    yield lambda out: bsq.int8_linear(x, z8(24, 64), one(24), out=out)
    q, w = bsq.mx_quantize(x, "mxfp8"), torch.zeros(2, 24, 64, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    yield lambda out: bsq.bs_gemm_grouped("mxfp8", *q, w, torch.zeros(2, 24, 2, dtype=torch.uint8, device="cuda"), off, out=out)


class TestOnTheGpu:
    pytestmark = gpu

    @pytest.mark.parametrize("which", range(3))
    def test_overlapping_rows_are_refused(self, which):
        call = list(_calls())[which]
        buf = torch.full((4 * 24,), 7.0, dtype=torch.bfloat16, device="cuda")
        for out in (buf[:24].expand(4, 24), buf.as_strided((4, 24), (23, 1))):
            with pytest.raises(bsq.BsqError):
                call(out)
        torch.cuda.synchronize()
        assert bool((buf == 7.0).all())
        assert call(buf.view(4, 24)).data_ptr() == buf.data_ptr() and bool((buf == 0).all())
