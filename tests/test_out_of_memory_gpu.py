"""An output that does not fit the memory: torch's own exception, which a program may catch."""
import pytest
import torch

import quantized_zero_communication_gb300 as zpp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_an_output_beyond_the_memory_raises_torchs_error():
    rows, vecs = 1 << 26, 65535  # 17.6 TB of fp32
    codes = torch.zeros(rows // 2, dtype=torch.uint8, device=DEV)
    x = torch.zeros(vecs, 1, device=DEV, dtype=torch.float16)
    with pytest.raises(torch.OutOfMemoryError):
        zpp.matvec_blockwise(codes, torch.ones(rows // 64, device=DEV), x, rows, 64, 4,
                             dtype=torch.float32)
