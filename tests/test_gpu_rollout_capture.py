"""The decode loop in CUDA graphs: one captured step, replayed, does what as many calls do."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_w4a4_quantized_quantize_gb300 import _lib, rollout
    assert _lib.device_status() == (0, 0)
    return rollout


def _state(batch):
    return [t.clone() for t in (batch.kv_len, batch.free_count, batch.q_off, batch.slots, batch.positions, batch.block_table)]


@pytest.mark.parametrize("steps", [1, 2, 5])
def test_a_captured_plan_advances(R, steps):
    """Every replay takes the lengths that the step before left: other slots each time, over borders of pages."""
    def batch():
        b = R.KVBatch(3, 16, 200, pages=40, max_new=24)
        b.plan(torch.tensor([15, 2, 0], dtype=torch.int32, device="cuda"))
        return b
    new = torch.tensor([1, 3, 1], dtype=torch.int32, device="cuda")
    plain, captured = batch(), batch()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured.plan(new)
    for _ in range(steps):
        plain.plan(new)
        g.replay()
        for a, b in zip(_state(plain), _state(captured)):
            assert torch.equal(a, b)
    assert captured.kv_len.tolist() == [15 + steps, 2 + 3 * steps, steps]


def test_lengths_stay_in_one_place(R):
    """A caller may keep the tensors: a plan changes what they hold, not which they are."""
    b = R.KVBatch(2, 16, 64, pages=8, max_new=8)
    kept, free = b.kv_len, b.free_count
    b.plan(torch.tensor([3, 1], dtype=torch.int32, device="cuda"))
    assert kept.tolist() == [3, 1] and free.tolist() == [6]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.plan(torch.tensor([1, 1], dtype=torch.int32, device="cuda"), stream=side)
    side.synchronize()
    assert kept.tolist() == [4, 2] and b.kv_len.data_ptr() == kept.data_ptr()
