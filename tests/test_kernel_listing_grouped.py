"""The operand-timing checks of test_kernel_listing on the expert-grouped 256 x 256
kernels, whose MFMAs are inline assembly too: the grouped instantiations of the
register-expansion NVFP4 GEMM and of the four-wave MX GEMM.  No GPU is needed;
skipped without hipcc."""

import pytest

from test_kernel_listing import _check_kernels, _compile, _functions


@pytest.mark.parametrize("source,kernel,suffixes", [
    ("bsq_gemm_nvfp4_rx.hip", "k_gemm_nvfp4_rx", ["ILb0ELi1E", "ILb0ELi2E"]),                       # rows, wgrad
    ("bsq_gemm_mx_rx.hip", "k_gemm_mx_grouped_rx", ["ILi1ELi1E", "ILi1ELi2E", "ILi2ELi1E", "ILi2ELi2E"]),
])
def test_grouped_mfma_operand_timing(source, kernel, suffixes):
    funcs = _functions(_compile(source), kernel)
    for s in suffixes:
        one = {n: b for n, b in funcs.items() if kernel + s in n}
        assert len(one) == 1, (s, list(funcs))
        _check_kernels(one)
