"""The rollout's decode step, composed from the C-ABI calls: a request's next tokens through attention over
the paged NVFP4 cache, routed experts and the head, with the log-probabilities the policy loss needs.

Weights are the rollout's NVFP4 operands (QUADS §3.2 Eq. (7)) against bf16 activations, which is the
learner's forward (Eq. (12)): a step has too few rows to gain from quantized activations, and its
log-probabilities then differ from the learner's (Eq. (2)) only by what the cache rounds.

    python -m nvfp4_w4a4_quantized_quantize_gb300.rollout          # a small random model answers prompts
"""
from __future__ import annotations

import argparse

import torch

from . import _lib as L
from .kvcache import KVBatch, KVCache
from .layers import Operand, quantize_weights


def _bf16(*shape, device="cuda"):
    return torch.empty(*shape, dtype=torch.bfloat16, device=device)


class W4A16Linear:
    """Y = X W-hat^T for a few rows: NVFP4 weights, bf16 activations.  `w` is a bf16 weight [N, K], or the
    operand that a RacLinear of the same layer keeps (its RAC tail is not read).  N of any size: the
    quantizer's rows are padded with zeros to a multiple of 128, which the product leaves out."""

    def __init__(self, w):
        if isinstance(w, Operand):
            self.op, self.N = w, w.rows
        else:
            self.N = w.shape[0]
            self.op = quantize_weights(torch.nn.functional.pad(w, (0, 0, 0, -self.N % 128)), 0)
        self.K = self.op.K

    def forward(self, x: torch.Tensor, out: torch.Tensor, stream=None):
        epi = L.NVQ_EPI_STORE_F32 if out.dtype is torch.float32 else L.NVQ_EPI_STORE
        L.nvfp4_gemv(x, self.op.codes, self.op.sf, self.op.sf_cols, self.op.tscale, self.N, self.K, out, epilogue=epi, stream=stream)
        return out


class W4A16Experts:
    """The routed SwiGLU experts of MoERacLayer for a few tokens: each (token, expert) pair is a row of two
    grouped products, so only the experts that have tokens are read.  w13 [E, 2I, H] and w2 [E, H, I] bf16,
    or the operands of a MoERacLayer (with E, I and H)."""

    def __init__(self, w13, w2, topk: int, E=None, inter=None, hidden=None):
        if isinstance(w13, Operand):
            self.E, self.I, self.H = E, inter, hidden
            self.w13, self.w2 = w13, w2
        else:
            self.E, self.I, self.H = w13.shape[0], w13.shape[1] // 2, w13.shape[2]
            self.w13, self.w2 = quantize_weights(w13, 0), quantize_weights(w2, 0)
        self.topk = topk

    def forward(self, x, topk_ids, topk_w, out, stream=None):
        """x [T, H] bf16, topk_ids int32 and topk_w fp32 [T, topk] -> out [T, H] bf16.  What lies between the calls is
        allocated, filled and released on the stream that they run on."""
        with torch.cuda.stream(stream):
            T, rows = x.shape[0], x.shape[0] * self.topk
            ids, w = topk_ids.view(-1), topk_w.view(-1)
            h, y = _bf16(rows, self.I, device=x.device), _bf16(rows, self.H, device=x.device)
            a, b = self.w13, self.w2
            L.nvfp4_gemv(x, a.codes, a.sf, a.sf_cols, a.tscale, 2 * self.I, self.H, h, ids=ids, groups=self.E, x_div=self.topk,
                         epilogue=L.NVQ_EPI_SWIGLU)
            L.nvfp4_gemv(h, b.codes, b.sf, b.sf_cols, b.tscale, self.H, self.I, y, ids=ids, groups=self.E,
                         epilogue=L.NVQ_EPI_ROW_SCALE, row_w=w)
            row_of = torch.arange(rows, dtype=torch.int64, device=x.device)
            L.moe_combine(y, row_of, T, self.topk, self.H, out)
        return out


class RolloutLayer:
    """Attention and experts with residuals; wqkv [(heads + 2 kv_heads) * head_dim, H], wo [H, heads * head_dim],
    router [E, H] bf16.  Rows are normalized (root mean square) before each half."""

    def __init__(self, wqkv, wo, router, w13, w2, heads: int, kv_heads: int, topk: int, cache: KVCache):
        self.heads, self.kv_heads, self.cache, self.topk = heads, kv_heads, cache, topk
        self.qkv, self.o, self.router = W4A16Linear(wqkv), W4A16Linear(wo), router
        self.experts = W4A16Experts(w13, w2, topk)

    def forward(self, x: torch.Tensor, batch: KVBatch, max_q: int):
        T, H, D = x.shape[0], self.heads, self.cache.head_dim
        qkv = self.qkv.forward(_normalized(x), _bf16(T, self.qkv.N)).view(T, -1, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + self.kv_heads], qkv[:, H + self.kv_heads:]
        L.nvfp4_kv_append(self.cache, k, v, batch.slots[:T])
        att = _bf16(T, H, D)
        L.nvfp4_kv_attention(self.cache, q, batch.kv_len, batch.block_table, att, batch.workspace, q_off=batch.q_off, max_q=max_q)
        x = x + self.o.forward(att.view(T, H * D), _bf16(*x.shape))
        n = _normalized(x)
        w, ids = torch.topk(torch.softmax((n @ self.router.t()).float(), -1), self.topk)
        w = w / w.sum(-1, keepdim=True)
        return x + self.experts.forward(n, ids.int(), w.contiguous(), _bf16(*x.shape))


def _normalized(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class RolloutModel:
    """Embedding, layers and head.  `step` takes every request's new tokens (a prompt, one token, or none)."""

    def __init__(self, embedding: torch.Tensor, layers: list, head: torch.Tensor):
        self.embedding, self.layers, self.head = embedding, layers, W4A16Linear(head)

    def step(self, batch: KVBatch, tokens: torch.Tensor, new_tokens, max_q: int = None):
        """tokens int64 [sum of new_tokens], request by request -> fp32 logits [tokens, V].  new_tokens: a count for each
        request, as a list, or as an int32 tensor on the device with max_q, a bound of the counts (such a step can be
        captured in a CUDA graph; rows of tokens beyond the counts' sum hold anything)."""
        if isinstance(new_tokens, torch.Tensor):
            if max_q is None or not tokens.numel():
                raise ValueError("new_tokens: counts on the device need max_q, a bound of them, and tokens, one at least")
        else:
            if not new_tokens or min(new_tokens) < 0 or not tokens.numel() or sum(new_tokens) != tokens.numel():
                raise ValueError(f"new_tokens: expected counts that add up to the {tokens.numel()} tokens, one at least, got {new_tokens}")
            max_q = max(new_tokens)
            new_tokens = torch.tensor(new_tokens, dtype=torch.int32, device=tokens.device)
        batch.plan(new_tokens)
        x = self.embedding[tokens]
        for layer in self.layers:
            x = layer.forward(x, batch, max_q)
        return self.head.forward(_normalized(x), torch.empty(x.shape[0], self.head.N, dtype=torch.float32, device=x.device))

    def answer(self, batch: KVBatch, prompts: list, steps: int, top_n: int = 4):
        """Greedy answers: (tokens, their log-probabilities, entropies) as [requests, steps] tensors."""
        if not all(p.numel() for p in prompts):
            raise ValueError("prompts: a request needs a token at least to continue from, its prompt is empty")
        dev, B = self.embedding.device, len(prompts)
        tokens, new = torch.cat(prompts), [p.numel() for p in prompts]
        kept = []
        for _ in range(steps):
            logits = self.step(batch, tokens, new)
            last = (batch.q_off[1:].long() - 1)  # each request's newest row
            logits = logits[last].contiguous()
            f32 = dict(dtype=torch.float32, device=dev)
            entropy, ids = torch.empty(B, **f32), torch.empty(B, top_n, dtype=torch.int32, device=dev)
            lps = torch.empty(B, top_n, **f32)
            L.token_logprobs(logits, entropy=entropy, top_ids=ids, top_logprobs=lps)
            tokens, new = ids[:, 0].long(), [1] * B
            kept.append((tokens, lps[:, 0], entropy))
        return tuple(torch.stack(c, 1) for c in zip(*kept))


def random_model(hidden=512, layers=2, heads=8, kv_heads=2, head_dim=64, experts=8, topk=2, inter=256, vocab=5000, page_size=16,
                 pages=256, seed=0, device="cuda") -> RolloutModel:
    g = torch.Generator(device=device).manual_seed(seed)

    def w(*shape, gain=1.0):
        return torch.randn(*shape, device=device, generator=g).mul_(gain * shape[-1] ** -0.5).bfloat16()
    stack = []
    for _ in range(layers):
        cache = KVCache.empty(pages, kv_heads, page_size, head_dim, k_amax=6.0, v_amax=6.0, device=device)
        stack.append(RolloutLayer(w((heads + 2 * kv_heads) * head_dim, hidden), w(hidden, heads * head_dim), w(experts, hidden),
                                  w(experts, 2 * inter, hidden), w(experts, hidden, inter), heads, kv_heads, topk, cache))
    return RolloutModel(w(vocab, hidden, gain=hidden ** 0.5), stack, w(vocab, hidden, gain=4.0))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=20, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args()
    model = random_model()
    vocab = model.embedding.shape[0]
    batch = KVBatch(a.requests, 16, a.prompt + a.steps, pages=256, max_new=a.requests * a.prompt)
    prompts = [torch.randint(0, vocab, (1 + i % a.prompt,), device="cuda") for i in range(a.prompt - a.requests, a.prompt)]
    tokens, logprobs, entropy = model.answer(batch, prompts, a.steps)
    status, where = L.device_status()
    if status:
        raise RuntimeError(f"device status {L.STATUS_NAMES.get(status, status)} at {where}")
    for r in range(a.requests):
        print(f"request {r}: prompt of {prompts[r].numel()} tokens, answer {tokens[r].tolist()}, log-probability "
              f"{float(logprobs[r].sum()):.3f}, mean entropy {float(entropy[r].mean()):.3f}")


if __name__ == "__main__":
    main()
