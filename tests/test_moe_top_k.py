"""The experts' top_k in the binding: whole numbers of any type, no fractions (no GPU needed)."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_05_b200 as q

M, E, H, F = 3, 4, 128, 64


def call(top_k):
    gu = q.QuantizedWeight.empty(E * 2 * F, H, True, "cpu")
    dn = q.QuantizedWeight.empty(E * H, F, True, "cpu")
    zeros = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    return q.nf4_moe_fwd(gu, dn, zeros(M, H), zeros(E, H), top_k)


@pytest.mark.parametrize("top_k", [2.7, 0.5, "2", np.float64(1.25), torch.tensor(1.5)])
def test_what_is_no_integer_is_refused(top_k):
    with pytest.raises(ValueError, match="top_k must be an integer"):
        call(top_k)


@pytest.mark.parametrize("top_k", [2, 2.0, np.int64(2), np.int32(2), torch.tensor(2)])
def test_integers_of_any_type_are_taken(top_k):
    with pytest.raises(ValueError, match="CUDA tensors"):         # every other check has passed
        call(top_k)
