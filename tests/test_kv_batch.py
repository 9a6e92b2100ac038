"""KVBatch's own checks, on the CPU."""
import pytest
import torch

from nvfp4_w4a4_quantized_quantize_gb300.kvcache import KVBatch


@pytest.mark.parametrize("n", [0, 1, 2, 4])
def test_plan_needs_a_count_for_every_request(n):
    """With fewer the others' lengths and query offsets would be those of an earlier step."""
    batch = KVBatch(3, 16, 64, pages=8, max_new=8, device="cpu")
    batch.kv_len.copy_(torch.tensor([5, 6, 7]))
    with pytest.raises(ValueError, match="3 requests"):
        batch.plan(torch.ones(n, dtype=torch.int32))
    assert batch.kv_len.tolist() == [5, 6, 7] and batch.free_count.tolist() == [8]
