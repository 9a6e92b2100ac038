"""Log-probabilities of given tokens with their entropy, for the policy loss (QUADS Eq. (2) compares
the rollout's with the trainer's), as an autograd node over token_logprobs and its backward."""
from __future__ import annotations

import torch

from . import _lib as L


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, scale):
        z, t = logits.detach().reshape(-1, logits.shape[-1]), targets.reshape(-1).contiguous()
        if z.stride(-1) != 1:
            z = z.contiguous()
        logprob, entropy, lse = (torch.empty(z.shape[0], dtype=torch.float32, device=z.device) for _ in range(3))
        L.token_logprobs(z, t, logprob, entropy, lse, scale=scale)
        ctx.save_for_backward(logits, z, t, lse, entropy)
        ctx.scale = scale
        return logprob.view(targets.shape), entropy.view(targets.shape)

    @staticmethod
    def backward(ctx, g_logprob, g_entropy):
        if not ctx.needs_input_grad[0]:
            return None, None, None
        return _Gradient.apply(*ctx.saved_tensors, g_logprob, g_entropy, ctx.scale), None, None


class _Gradient(torch.autograd.Function):
    """The gradient as a node of its own, on the logits and the incoming gradients: under create_graph its result then
    requires a gradient, which no entry computes and which raises.  (once_differentiable looks at the incoming
    gradients alone, and leaves a penalty on the gradient of a plain sum out without an error.)"""

    @staticmethod
    def forward(ctx, logits, z, t, lse, entropy, g_logprob, g_entropy, scale):
        grad = torch.empty(z.shape, dtype=z.dtype, device=z.device)
        glp, gh = (g.reshape(-1).float().contiguous() for g in (g_logprob, g_entropy))
        L.token_logprobs_backward(z, t, lse, entropy, glp, gh, grad, scale=scale)
        return grad.view(logits.shape)

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("token_logprobs has no second derivative: its node is once_differentiable")


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, temperature: float = 1.0):
    """(logprob, entropy), float32 of targets' shape, of logits [..., V] (bf16 or fp32) at `temperature`; rows with a
    negative target give 0 and take no gradient.  Differentiable in the logits, once: a second derivative raises."""
    return _TokenLogprobs.apply(logits, targets, 1.0 / temperature)
