"""The operand-timing checks of test_kernel_listing on the LDS-ring kernels of the
8-bit integer products and of the orthogonalisation's FP16 products whose MFMAs are
inline assembly too (tiles of 192 and 256, and of 128 with two buffers; the others'
MFMAs are the compiler's).  A copy between accumulators counts as a read of the one and
a write of the other.  No GPU is needed; skipped without hipcc."""

import re

import pytest

from test_kernel_listing import _compile, _functions, _instructions, hazards


def _copies_split(lines):
    """Each accumulator copy as the read and the write that the checks know."""
    out = []
    for line in lines:
        m = re.match(r"\s*v_accvgpr_mov_b32 (a\d+), (a\d+)", line)
        if m:
            out += [f"\tv_accvgpr_read_b32 v255, {m.group(2)}", f"\tv_accvgpr_write_b32 {m.group(1)}, v255"]
        else:
            out.append(line)
    return out


def test_copies_are_checked():
    mfma = "\tv_mfma_f32_16x16x32_f16 a[4:7], v[0:3], v[4:7], a[4:7]"
    assert len(hazards(_copies_split([mfma, "\tv_accvgpr_mov_b32 a9, a5"]))) == 1
    assert len(hazards(_copies_split(["\tv_accvgpr_mov_b32 a5, a9", mfma]))) == 1
    assert hazards(_copies_split([mfma, "\tv_accvgpr_mov_b32 a9, a15"])) == []


@pytest.mark.parametrize("source", ["bsq_int8.hip", "bsq_ortho.hip"])
def test_ring_mfma_operand_timing(source):
    funcs = _functions(_compile(source), "k_nt_ring")
    asm = {n: b for n, b in funcs.items() if re.search(r"k_nt_ringILi\dELi(8ELi2|6ELi3|4ELi2)E", n)}
    assert len(asm) >= 6 and len(funcs) > len(asm), list(funcs)
    for name, body in asm.items():
        assert any(mn.startswith("v_mfma") for mn, _ in _instructions(body)), name
        assert not hazards(_copies_split(body)), (name, hazards(_copies_split(body))[:5])
