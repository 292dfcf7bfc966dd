"""Arguments that a call would have answered wrongly."""
import numpy as np
import pytest
import torch

import huffman_decode_canonical_b200 as entro


@pytest.mark.parametrize("zero", [3.5, 3.0, np.float32(2), float("nan"), "3"])
def test_a_zero_point_is_a_whole_number(zero):
    """(Fractions were cut off.)"""
    x = entro.QuantTokens(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), torch.zeros(4, dtype=torch.int32))
    w = torch.zeros(8, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="whole number"):
        entro.matmul_i8(x, w, 1.0, zero)
    for whole in (3, np.int64(3), np.int32(-3)):  # as far as the refusal of CPU tensors
        with pytest.raises(ValueError, match="CUDA"):
            entro.matmul_i8(x, w, 1.0, whole)


def test_prompt_attention_does_not_write_its_inputs():
    """(Other blocks still read keys and values; queries are read again where a sequence's values hold an infinity.)"""
    q, k, v = (torch.zeros(6, 4, 64, dtype=torch.bfloat16) for _ in range(3))
    cu = torch.tensor([0, 6], dtype=torch.int32)
    for out in (q, k, v, q.view(6, 4, 64)):
        with pytest.raises(ValueError, match="must not be"):
            entro.attention_prompt(q, k, v, cu, out=out)
    both = torch.zeros(6, 8, 64, dtype=torch.bfloat16)  # beside each other in one buffer: as far as the refusal of CPU tensors
    with pytest.raises(ValueError, match="CUDA"):
        entro.attention_prompt(both[:, :4], k, v, cu, out=both[:, 4:])
