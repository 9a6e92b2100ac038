"""Keys and values that are not finite, in the cache: the block quantizer gives finite codes and scales for them, so what a
query does not see cannot reach it.

Tolerance, by test_gpu_kv_attention.py: an output is off by (2 d + 2^-10) sum p|v| + 2^-8 |out| and an lse by d + 2^-20 (1 +
|lse|), d = 2^-17 scale sum|q||k| <= 2^-13 here and |v| <= 5; two runs differ by twice that.  (Not the same bits: rows of a
tile move their running maxima together.)"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("whole", [False, True])
def test_an_unseen_tokens_values_do_not_matter(bad, whole):
    """Three new tokens, the last of which is not finite, in one place or throughout: the two before it are as they were."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_w4a4_quantized_quantize_gb300 import _lib as L
    from nvfp4_w4a4_quantized_quantize_gb300.kvcache import KVBatch, KVCache
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(40, 2, 64, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn(3, 8, 64, device="cuda", generator=g).bfloat16()
    outs = []
    for x in (None, bad):
        cache = KVCache.empty(8, 2, 16, 64, k_amax=4.0, v_amax=4.0)
        batch = KVBatch(1, 16, 64, pages=8, max_new=40)
        kk, vv = k.clone(), v.clone()
        if x is not None:
            for t in (kk, vv):
                t[39, :, slice(None) if whole else 5] = x
        for first, n in ((0, 37), (37, 3)):
            batch.plan(torch.tensor([n], dtype=torch.int32, device="cuda"))
            L.nvfp4_kv_append(cache, kk[first:first + n], vv[first:first + n], batch.slots[:n])
        for sf in (cache.k_sf, cache.v_sf):
            assert ((sf & 0x7F) != 0x7F).all()
        out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
        L.nvfp4_kv_attention(cache, q, batch.kv_len, batch.block_table, out, batch.workspace, q_off=batch.q_off, max_q=3, lse=lse)
        assert L.device_status() == (0, 0)
        outs.append((out, lse))
    (a, la), (b, lb) = outs
    tol = 2 * ((2 ** -12 + 2 ** -10) * 5 + 2 ** -8 * a[:2].abs().double())
    assert ((a[:2].double() - b[:2].double()).abs() <= tol).all()
    assert ((la[:2] - lb[:2]).abs() <= 2 * (2 ** -13 + 2 ** -20 * (1 + la[:2].abs()))).all()
    assert b.isfinite().all() and lb.isfinite().all()
