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


def test_a_captured_step_answers_like_the_loop(R):
    """Embedding to the choice of the next token in one graph, replayed step after step."""
    from nvfp4_w4a4_quantized_quantize_gb300 import _lib as L
    steps = 20  # past a page's border
    model = R.random_model(layers=2, vocab=1000, pages=64)
    prompts = [torch.tensor([5, 9, 2], device="cuda"), torch.tensor([700], device="cuda"), torch.arange(15, device="cuda")]
    want, lps, _ = model.answer(R.KVBatch(3, 16, 64, pages=64, max_new=40), prompts, steps)
    for layer in model.layers:
        for t in (layer.cache.k_codes, layer.cache.k_sf, layer.cache.v_codes, layer.cache.v_sf):
            t.zero_()

    batch = R.KVBatch(3, 16, 64, pages=64, max_new=40)
    logits = model.step(batch, torch.cat(prompts), [p.numel() for p in prompts])
    token = logits[batch.q_off[1:].long() - 1].argmax(-1)
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    ids, lp = torch.empty(3, 1, dtype=torch.int32, device="cuda"), torch.empty(3, 1, device="cuda")

    def step():
        L.token_logprobs(model.step(batch, token, one, max_q=1), top_ids=ids, top_logprobs=lp)
        token.copy_(ids[:, 0])

    state = _state(batch) + [token.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the libraries' first calls are not for a capture
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip((batch.kv_len, batch.free_count, batch.q_off, batch.slots, batch.positions, batch.block_table, token), state):
        t.copy_(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    got, got_lps = [token.clone()], []
    for _ in range(steps - 1):
        g.replay()
        got.append(token.clone())
        got_lps.append(lp[:, 0].clone())
    assert L.device_status() == (0, 0)
    assert torch.equal(torch.stack(got, 1), want)
    assert torch.equal(torch.stack(got_lps, 1), lps[:, 1:])
    assert batch.kv_len.tolist() == [p.numel() + steps - 1 for p in prompts]
