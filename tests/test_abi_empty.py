"""Zero-size calls of the quantizers with the null pointers that empty tensors have
are BSQ_OK, as the header says of every entry point (no GPU: nothing is launched)."""

import os

import pytest

import fp8_quantized_gemm_amd as bsq

pytestmark = pytest.mark.skipif(not os.path.exists(bsq.LIB_PATH),
                                reason="libbsq.so not built (run __graft_entry__.build())")

FAKE = 0x1000000       # an aligned address, never dereferenced


@pytest.mark.parametrize("rows,cols", [(0, 64), (64, 0), (0, 0)])
def test_empty_tensors_have_null_pointers(rows, cols):
    L = bsq.lib()
    for fmt in (0, 1, 2):
        assert L.quantize_transpose(None, rows, cols, fmt, 1, 0, 0, 0, 0, 0, *[None] * 7) == bsq.BSQ_OK
    assert L.quantize_transpose_amax(None, rows, cols, 1, 0, 0, 0, 0, 0, FAKE, FAKE, *[None] * 5) == bsq.BSQ_OK
    assert L.quantize_transpose_amax(None, rows, cols, 16, 0, 0, 0, 0, 0, FAKE, FAKE, *[None] * 5) == bsq.BSQ_OK
    # the other checks still hold
    assert L.quantize_transpose_amax(None, rows, cols, 2, 0, 0, 0, 0, 0, FAKE, FAKE, *[None] * 5) == bsq.BSQ_EINVAL
    assert L.quantize_transpose_amax(None, 16, 16, 1, 0, 0, 0, 0, 0, FAKE, FAKE, *[None] * 5) == bsq.BSQ_EINVAL
    assert L.fp8_quantize_transpose(None, rows, cols, None, None, None, None) == bsq.BSQ_EINVAL   # amax is required
