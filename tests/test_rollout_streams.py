"""Streams of the decode step's layers: on the CPU with the entries that launch kernels stood in for, and on a GPU."""
import contextlib

import pytest
import torch

from nvfp4_w4a4_quantized_quantize_gb300 import rollout


def test_experts_keep_to_the_stream_they_are_given(monkeypatch):
    """What the experts allocate and fill between their calls belongs to the stream that the calls run on."""
    inside, made, calls = [None], [], []

    @contextlib.contextmanager
    def stream(s):
        before, inside[0] = inside[0], s if s is not None else inside[0]
        yield
        inside[0] = before

    def recorded(f):
        def g(*a, **kw):
            made.append(inside[0])
            return f(*a, **kw)
        return g

    def entry(*a, stream=None, **kw):
        calls.append(stream if stream is not None else inside[0])
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("empty", "arange", "zeros"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    for name in ("nvfp4_gemv", "moe_combine"):
        monkeypatch.setattr(rollout.L, name, entry)
    op = rollout.Operand(None, None, 4, None, 128, 64, 0)
    experts = rollout.W4A16Experts(op, op, 2, E=4, inter=64, hidden=64)
    x, out = torch.ones(3, 64), torch.ones(3, 64)
    for want in ("side", None):
        made.clear()
        calls.clear()
        experts.forward(x, torch.ones(3, 2, dtype=torch.int32), torch.ones(3, 2), out, stream=want)
        assert len(calls) == 3 and made and set(made) == set(calls) == {want}


@pytest.mark.gpu
def test_experts_on_a_side_stream_beside_other_work():
    """The current stream takes and fills memory of the same sizes right after each call."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    g = torch.Generator(device="cuda").manual_seed(1)
    E, H, I, T, topk = 8, 256, 128, 24, 2
    w13 = torch.randn(E, 2 * I, H, device="cuda", generator=g).mul_(0.06).bfloat16()
    w2 = torch.randn(E, H, I, device="cuda", generator=g).mul_(0.06).bfloat16()
    experts = rollout.W4A16Experts(w13, w2, topk)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    ids = torch.rand(T, E, device="cuda", generator=g).argsort(-1)[:, :topk].int().contiguous()
    w = torch.rand(T, topk, device="cuda", generator=g)
    want = experts.forward(x, ids, w, torch.empty_like(x))
    side = torch.cuda.Stream()
    outs = [torch.full_like(x, 9.0) for _ in range(50)]
    side.wait_stream(torch.cuda.current_stream())
    for out in outs:
        experts.forward(x, ids, w, out, stream=side)
        for shape, dtype in (((T * topk, I), torch.bfloat16), ((T * topk, H), torch.bfloat16), ((T * topk,), torch.int64)):
            torch.empty(*shape, dtype=dtype, device="cuda").fill_(-1)
    side.synchronize()
    for out in outs:
        assert torch.equal(out, want)
    assert rollout.L.device_status() == (0, 0)
