"""What RolloutModel's step and answer refuse, on the CPU."""
import pytest
import torch

from nvfp4_w4a4_quantized_quantize_gb300 import rollout


def _model():
    class Stub(rollout.RolloutModel):
        def __init__(self):
            self.embedding, self.layers = torch.ones(9, 4), []
    return Stub()


def test_answers_need_a_prompt():
    """A request without tokens has no newest row to continue from."""
    with pytest.raises(ValueError, match="prompt"):
        _model().answer(None, [torch.tensor([1, 2]), torch.tensor([], dtype=torch.int64)], 3)


@pytest.mark.parametrize("tokens,new", [(3, [1, 1]), (3, [2, 2]), (0, [0, 0]), (2, [3, -1]), (0, [])])
def test_steps_need_as_many_tokens_as_they_count(tokens, new):
    with pytest.raises(ValueError, match="new_tokens"):
        _model().step(None, torch.ones(tokens, dtype=torch.int64), new)


def test_a_step_with_counts_on_the_device_needs_their_bound():
    with pytest.raises(ValueError, match="max_q"):
        _model().step(None, torch.ones(2, dtype=torch.int64), torch.ones(2, dtype=torch.int32))
