"""The log-probabilities' autograd node on the CPU: the entries that launch kernels are stood in for."""
import pytest
import torch

from nvfp4_w4a4_quantized_quantize_gb300 import logprobs


class _Entries:
    """token_logprobs and its backward in torch."""

    @staticmethod
    def token_logprobs(z, t, logprob, entropy, lse, scale=1.0):
        lp = torch.log_softmax(z.float() * scale, -1)
        lse.copy_(torch.logsumexp(z.float() * scale, -1))
        logprob.copy_(lp.gather(1, t[:, None]).squeeze(1))
        entropy.copy_(-(lp.exp() * lp).sum(-1))

    @staticmethod
    def token_logprobs_backward(z, t, lse, entropy, glp, gh, grad, scale=1.0):
        lp = z * scale - lse[:, None]
        grad.copy_(-lp.exp() * (glp[:, None] + gh[:, None] * (lp + entropy[:, None])) * scale)
        grad.scatter_add_(1, t[:, None], glp[:, None] * scale)


def test_second_derivatives_of_log_probabilities_are_refused(monkeypatch):
    """The node has a gradient, but not that gradient's gradient: a penalty on it raises, and is not left out."""
    monkeypatch.setattr(logprobs, "L", _Entries)
    z = torch.randn(3, 7, requires_grad=True)
    t = torch.tensor([1, 0, 6])
    lp, h = logprobs.token_logprobs(z, t)
    (g,) = torch.autograd.grad((lp + 0.1 * h).sum(), z, create_graph=True)
    ls = torch.log_softmax(z.detach().requires_grad_(True), -1)
    assert (lp - ls.gather(1, t[:, None]).squeeze(1)).abs().max() < 1e-6
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (lp.sum() + g.square().sum()).backward()


def test_a_graph_of_the_gradient_that_is_not_used_changes_nothing(monkeypatch):
    monkeypatch.setattr(logprobs, "L", _Entries)
    t = torch.tensor([2, 2, 5])
    grads = []
    for create in (False, True):
        z = torch.linspace(-1, 1, 21).view(7, 3).t().requires_grad_(True)  # rows that are not contiguous
        lp, h = logprobs.token_logprobs(z, t, temperature=0.5)
        grads.append(torch.autograd.grad(lp.sum() - h.sum(), z, create_graph=create)[0])
    assert torch.equal(grads[0], grads[1].detach()) and grads[1].requires_grad and not grads[0].requires_grad
    w = torch.ones(3, requires_grad=True)  # weights of the loss that take a gradient themselves
    z = torch.randn(3, 7, requires_grad=True)
    (g,) = torch.autograd.grad((w * logprobs.token_logprobs(z, t)[0]).sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()
