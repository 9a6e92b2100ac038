"""Every row of the decode step against the plain model in 64 bits: with as many experts as are chosen no row is
excused, and where the router chooses, none whose choice is clear.

Tolerance, before any run: that of test_gpu_rollout.py, 2e-2 of the row's norm (bf16 roundings come to 1e-2).  A
router's logits are products of a row of norm sqrt(hidden), off by at most 1e-2 of its norm in a direction that has
nothing to do with the router's rows of norm 1: about 1e-2 each, 1.4e-2 their difference, and each is rounded to
bf16, 2^-7 at a size of 4.  A choice is clear where the logits on either side of it differ by more than 6 times
1.4e-2 and twice 2^-7: 0.1, and a little."""
import math

import pytest
import torch

from tests.test_gpu_rollout import _cached, _norm, _weights

pytestmark = pytest.mark.gpu

TOL, CLEAR = 2e-2, 0.12


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_w4a4_quantized_quantize_gb300 import rollout
    return rollout


def _plain(model, batch, tokens, new):
    """Logits of the plain model on a step that has run, and the least gap at a row's choice of experts."""
    x = model.embedding[tokens].double()
    gap = torch.full((x.shape[0],), math.inf, dtype=torch.float64, device="cuda")
    lens, first = batch.kv_len.tolist(), batch.q_off.tolist()
    for layer in model.layers:
        H, KV, D = layer.heads, layer.kv_heads, layer.cache.head_dim
        q = (_norm(x) @ _weights(layer.qkv.op, 1)[0].t())[:, :H * D].view(-1, KV, H // KV, D)
        att = torch.zeros(x.shape[0], KV, H // KV, D, dtype=torch.float64, device="cuda")
        for b, n in enumerate(new):
            K, V = _cached(layer.cache, batch, b, lens[b])
            for i in range(n):
                hi = lens[b] - n + i + 1
                z = torch.einsum("kgd,jkd->kgj", q[first[b] + i], K[:hi]) / math.sqrt(D)
                att[first[b] + i] = torch.einsum("kgj,jkd->kgd", torch.softmax(z, -1), V[:hi])
        x = x + att.flatten(1) @ _weights(layer.o.op, 1)[0].t()
        n = _norm(x)
        r = n @ layer.router.double().t()
        E, k, inter = layer.experts.E, layer.topk, layer.experts.I
        if k < E:
            z = torch.sort(r, -1, descending=True).values
            gap = torch.minimum(gap, z[:, k - 1] - z[:, k])
        w, ids = torch.topk(torch.softmax(r, -1), k)
        p = torch.zeros_like(r).scatter_(1, ids, w / w.sum(-1, keepdim=True))
        gu = torch.einsum("enh,th->ten", _weights(layer.experts.w13, E), n)
        h = torch.nn.functional.silu(gu[..., :inter]) * gu[..., inter:]
        x = x + torch.einsum("te,eni,tei->tn", p, _weights(layer.experts.w2, E), h)
    return _norm(x) @ _weights(model.head.op, 1)[0].t(), gap


def _rows(R, model, seed):
    """(share of the norm that each row is off by, its gap) over prompts, single tokens, idle requests and drafts."""
    from nvfp4_w4a4_quantized_quantize_gb300 import _lib as L
    batch = R.KVBatch(3, 16, 80, pages=64, max_new=64)
    g = torch.Generator(device="cuda").manual_seed(seed)
    off, gaps = [], []
    for new in ([17, 1, 30], [1, 1, 1], [1, 0, 1], [4, 1, 2], [0, 0, 1], [1, 1, 1]):
        tokens = torch.randint(0, 512, (sum(new),), device="cuda", generator=g)
        logits = model.step(batch, tokens, new).double()
        assert L.device_status() == (0, 0)
        ref, gap = _plain(model, batch, tokens, new)
        off.append((logits - ref).norm(dim=-1) / ref.norm(dim=-1))
        gaps.append(gap)
    return torch.cat(off), torch.cat(gaps)


@pytest.mark.parametrize("experts", [1, 2, 4])
def test_every_row_where_all_experts_are_chosen(R, experts):
    off, _ = _rows(R, R.random_model(layers=2, experts=experts, topk=experts, vocab=512, pages=64, seed=experts), experts)
    assert off.numel() == 64 and (off < TOL).all(), off


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_every_row_whose_experts_are_clear(R, seed):
    """Of eight experts two, in one layer: most choices are clear."""
    off, gap = _rows(R, R.random_model(layers=1, experts=8, topk=2, vocab=512, pages=64, seed=seed), seed)
    clear = gap > CLEAR
    assert clear.float().mean() >= 0.5 and (off[clear] < TOL).all(), off[clear]
