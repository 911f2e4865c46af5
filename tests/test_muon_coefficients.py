"""How the coefficients of the Newton-Schulz steps are taken (no GPU)."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amd as bsq


def _taken(steps, coefs):
    return list(bsq._coefs(steps, bsq._coef_key(coefs)))


def test_tensors_and_arrays_by_their_values():
    one, two = [1.0, 2.0, 3.0], [[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]]
    for kind in (list, tuple, np.array, torch.tensor, lambda v: iter(v)):
        assert _taken(2, kind(one)) == one * 2
        assert _taken(2, kind(two)) == two[0] + two[1]
    assert _taken(1, [torch.tensor(v) for v in one]) == one


def test_a_tensor_changed_in_place():
    """The second call's coefficients are those that the tensors hold then."""
    for make in (lambda: tuple(torch.tensor(v) for v in (1.0, 2.0, 3.0)), lambda: torch.tensor([1.0, 2.0, 3.0]),
                 lambda: [list(torch.tensor([1.0, 2.0, 3.0]))]):
        c = make()
        assert _taken(1, c) == [1, 2, 3]
        (c[0][0] if isinstance(c[0], list) else c[0]).fill_(7.0)
        assert _taken(1, c) == [7, 2, 3]


def test_refused():
    for c in (None, 3.0, "abc", ("a", 1, 2), (1, 2), [[1, 2, 3], 4], torch.zeros(2, 3), np.zeros((1, 3, 1)), (1j, 2, 3)):
        with pytest.raises(ValueError):
            _taken(1, c)
