"""token_logprobs_backward where the row's lse is so large that fp32 cannot hold the logarithm of its sum: rows
shifted by a constant, masked throughout by a large negative number, or at a low temperature.  The weights p
do not depend on a shift, so neither does the gradient.

Tolerances, before any run.  With z = scale * logit - lse as fp32 gives it and S = sum exp(z), p = exp(z) / S.
lse is off by its own rounding, at most 2^6 where |lse| < 2^31, and the terms that count lie within 2^6 of
the largest, so |z|, |log S| <= 2^7 and each of their fp32 roundings (z, its multiple of log2 e, log S, and
2^-22 of an exp2) moves a weight by at most 2^-16; four of them, and S off by as much again: 2^-13.  The slope
log p + H is off by 2^-15 of 2^7 at most; H itself by 2^-15 (1 + H).  A target's term: 2^-22.  bf16 results: 2^-8 of
each.  Sums of a row's p add up: 2^-12, with bf16 2^-8."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_w4a4_quantized_quantize_gb300 import _lib
    assert _lib.device_status() == (0, 0)
    return _lib


def _check(L, z, scale=1.0, in_place=False):
    T, V = z.shape
    f32 = dict(dtype=torch.float32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(V)
    # targets among the likely: the largest of a few random places of each row
    at = torch.randint(0, V, (T, 16), device="cuda", generator=g)
    t = at.gather(1, z.float().gather(1, at).argmax(-1, keepdim=True)).squeeze(1)
    lp, h, lse = (torch.empty(T, **f32) for _ in range(3))
    L.token_logprobs(z, t, lp, h, lse, scale=scale)
    zd = z.double() * float(torch.tensor(scale, dtype=torch.float32))
    ref = torch.log_softmax(zd, -1)
    p = ref.exp()
    l0 = torch.where(p > 0, ref, 0.0)
    H = -(p * l0).sum(-1, keepdim=True)
    weights = [(torch.ones(T, **f32), None), (torch.randn(T, generator=g, **f32), torch.randn(T, generator=g, **f32)),
               (None, torch.ones(T, **f32))]
    for glp, gh in weights:
        src = z.clone()
        out = src if in_place else torch.full_like(z, 7.0)
        L.token_logprobs_backward(src, t, lse, h, glp, gh, out, scale=scale)
        a, b = (torch.zeros(T, 1, dtype=torch.float64, device="cuda") if w is None else w.double()[:, None] for w in (glp, gh))
        want = -p * (a + b * (l0 + H))
        tol = p * (a.abs() + b.abs() * (l0.abs() + H)) * 2 ** -13 + p * b.abs() * (2 ** -8 + 2 ** -15 * (1 + H)) + 1e-37
        want.scatter_add_(1, t[:, None], a)
        tol.scatter_add_(1, t[:, None], 2 ** -22 * a.abs())
        if z.dtype is torch.bfloat16:
            tol += 2 ** -8 * want.abs()
        bad = (out.double() - scale * want).abs() > scale * tol
        assert not bad.any(), (out[bad][:4], (scale * want)[bad][:4], (scale * tol)[bad][:4])
        if gh is None:  # the sum of p, from the gradient of the target's log-probability at all other places
            total = -out.double().scatter(1, t[:, None], 0.0).sum(-1) / scale + p.gather(1, t[:, None]).squeeze(1)
            assert ((total - 1.0).abs() <= (2 ** -8 if z.dtype is torch.bfloat16 else 2 ** -12)).all(), total
    assert L.device_status() == (0, 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [7, 1003, 32000, 131072])
@pytest.mark.parametrize("offset", [250.0, 260.0, 1e3, 3e4, 1e6, 1e7, 3e7, 1e8, 1e9, 1.5e9, 2.2e9])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_shifted_rows(L, dtype, V, offset, sign):
    """Constant rows, rows that vary (as far as the type can at that size), and constant rows masked in half."""
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.full((4, V), sign * offset, device="cuda")
    z[1] += torch.randn(V, device="cuda", generator=g).mul_(2.0)
    z[2, 1::2] = -math.inf
    z[3] += torch.randint(0, 3, (V,), device="cuda", generator=g) * offset * 2 ** -22
    _check(L, z.to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [30.0, 1e3, 1e5, 1e6, 1e8])
def test_low_temperatures(L, dtype, scale):
    """Ordinary logits at a temperature near zero: weights on the largest, or even over its ties."""
    z = torch.randn(5, 5003, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).mul_(3.0)
    z[1, 100:110] = 15.0
    z[2] = 11.0
    z[3] = -0.0078125
    _check(L, z.to(dtype), scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [1e3, -1e9])
def test_in_place_over_several_blocks(L, dtype, offset):
    """A row of many blocks' width, its gradient written over it; rows beside it of ordinary size, and more
    rows than the GPU holds at once."""
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(700, 40003, device="cuda", generator=g)
    z[::2] += offset
    _check(L, z.to(dtype), in_place=True)
