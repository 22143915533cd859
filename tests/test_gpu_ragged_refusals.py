"""Refusals of the ragged products that come before anything is allocated."""
import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [0, 1025, 5000])
def test_number_of_experts(E):
    """dw of 5000 experts would be 670 GB: a refusal, not a failed allocation."""
    x, dout = (torch.zeros((32, 8192), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    offs = torch.full((E,), 32, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(mx.MxError):
        mx.ragged_mm_wgrad(dout, x, offs)
    assert torch.cuda.max_memory_allocated() == before
