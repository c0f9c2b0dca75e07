"""An optimiser over more tensors than a call takes is refused when it is made, with the reason, and
not at its first step."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_call_takes(bits):
    with pytest.raises(ValueError, match="1025 tensors, at most 1024"):
        zpp.AdamW([torch.zeros(1)] * 1025, state_bits=bits)
