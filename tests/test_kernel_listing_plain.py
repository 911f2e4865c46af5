"""The operand-timing checks of test_kernel_listing on the LDS-ring kernels of the
8-bit integer products and of the orthogonalisation's FP16 products, whose MFMAs are
inline assembly too.  No GPU is needed; skipped without hipcc."""

import pytest

from test_kernel_listing import _check_kernels, _compile, _functions


@pytest.mark.parametrize("source", ["bsq_int8.hip", "bsq_ortho.hip"])
def test_ring_mfma_operand_timing(source):
    funcs = _functions(_compile(source), "k_nt_ring")
    assert funcs
    _check_kernels(funcs)
