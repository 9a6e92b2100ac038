"""nvfp4_kv_attention on prompts so long that the units of work pass 32 bits, and what it writes when an index is bad.

Tolerances are those of test_gpu_kv_attention.py, from the same reasoning; the sums of up to 500000 weights add
2^-20 relative (pieces and lanes sum at most 2^11 terms one after the other)."""
import math

import pytest
import torch

from tests.test_gpu_kv_attention import ERR_ARG, WHERE_ATTENTION, Case, L, _values, work  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def _check_rows(case, out, lse, picks, window=0):
    """Queries picks [(request, i)] against attention in 64 bits."""
    c = case.cache
    rows, heads, dim = case.q.shape
    G = heads // c.kv_heads
    first = case.q_off.tolist()
    scale = dim ** -0.5
    for b in sorted({b for b, _ in picks}):
        n, m = case.lens[b], case.n_q[b]
        j = torch.arange(n, device="cuda")
        pg, at = case.table[b, j // case.page].long(), j % case.page
        K = _values(c.k_codes[pg, :, at], c.k_sf[pg, :, at], c.k_tscale[0, 2].double()).transpose(0, 1)
        V = _values(c.v_codes[pg, :, at], c.v_sf[pg, :, at], c.v_tscale[0, 2].double()).transpose(0, 1)
        for i in (i for q, i in picks if q == b):
            t, hi = first[b] + i, n - m + i + 1
            lo = max(0, hi - window) if window else 0
            q = case.q[t].double().view(c.kv_heads, G, dim)
            z = q @ K[:, lo:hi].transpose(1, 2) * scale
            s = torch.logsumexp(z, -1)
            p = (z - s[..., None]).exp()
            d = 2 ** -17 * scale * (q.abs() @ K[:, lo:hi].abs().transpose(1, 2)).amax(-1) + 2 ** -21 * z.abs().amax(-1)
            o = p @ V[:, lo:hi]
            tol = (2 * d[..., None] + 2 ** -10 + 2 ** -20) * (p @ V[:, lo:hi].abs()) + 2 ** -8 * o.abs()
            assert ((out[t].double().view_as(o) - o).abs() <= tol).all(), (b, i)
            assert ((lse[t].double().view_as(s) - s).abs() <= d + 2 ** -19 * (1 + s.abs())).all(), (b, i)


@pytest.mark.parametrize("lens,n_q,heads", [([65535] * 9, [65535] * 9, 16), ([3, 500000, 70], [1, 34768, 2], 32)])
def test_units_of_work_beyond_32_bits(L, work, lens, n_q, heads):  # noqa: F811
    """Nine prompts of 65535 tokens, and one long piece of a prompt over 500000 keys: more than 2^31 units each.
    Every row is written; those looked at are right."""
    c = Case(lens, n_q, heads, 1, 64, 64, seed=1, extra_blocks=0)
    out, lse = torch.full_like(c.q, math.nan), torch.full(c.q.shape[:2], math.nan, device="cuda")
    L.nvfp4_kv_attention(c.cache, c.q, c.kv_len, c.table, out, work, q_off=c.q_off, max_q=max(n_q), lse=lse)
    assert L.device_status() == (0, 0)
    picks = [(b, i) for b in range(len(lens)) for i in sorted({0, 1, n_q[b] // 3, n_q[b] - 2, n_q[b] - 1}) if 0 <= i < n_q[b]]
    _check_rows(c, out, lse, picks)
    assert lse.isfinite().all() and out.isfinite().all()
    again = Case([40, 0, 7], [1, 1, 1], 8, 2, 64, 16, seed=2)  # the workspace is ready for the next call
    again.check(L, work)


def _bad(L, work, case):  # noqa: F811
    got = case.run(L, work)
    assert L.device_status() == (ERR_ARG, WHERE_ATTENTION)
    return got


def _same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("page", [-1, 99])
def test_a_page_outside_the_cache_reads_page_0(L, work, page):  # noqa: F811
    c = Case([112, 50], [2, 1], 4, 2, 64, 16, seed=3, extra_blocks=0)
    c.cache.k_sf[0], c.cache.v_sf[0] = 0x38, 0x38  # page 0 may be no request's: finite all the same
    c.table[0, 1] = 0
    want = c.run(L, work)
    assert L.device_status() == (0, 0)
    c.table[0, 1] = page
    _same(_bad(L, work, c), want)


def test_a_length_beyond_the_table_ends_at_the_table(L, work):  # noqa: F811
    c = Case([112, 50], [2, 1], 4, 2, 64, 16, seed=4, extra_blocks=0)
    want = c.check(L, work)
    c.kv_len[0] = 113
    _same(_bad(L, work, c), want)
    c.kv_len[0] = 2 ** 31 - 1
    _same(_bad(L, work, c), want)


def test_a_negative_length_is_an_empty_request(L, work):  # noqa: F811
    c = Case([0, 112], [1, 2], 4, 2, 64, 16, seed=5, extra_blocks=0)
    want = c.check(L, work)
    assert (want[0][0] == 0).all() and (want[1][0] == -math.inf).all()
    c.kv_len[0] = -5
    _same(_bad(L, work, c), want)


def test_bad_query_offsets_leave_the_requests_rows_unwritten(L, work):  # noqa: F811
    c = Case([100, 50, 30], [2, 1, 3], 4, 2, 64, 16, seed=6)
    c.check(L, work)
    full = c.q_off.clone()
    c.q_off[1] = 9  # request 0 leaves the query rows, request 1's offsets descend
    out, lse = _bad(L, work, c)
    assert (out[:3] == 9.0).all() and (lse[:3] == 9.0).all()
    c.q_off = full
    _check_rows(c, out, lse, [(2, i) for i in range(3)])
    c.n_q = [1, 1, 1]  # max_q of 1: requests 0 and 2 have more
    out, lse = _bad(L, work, c)
    assert (out[[0, 1, 3, 4, 5]] == 9.0).all() and (lse[[0, 1, 3, 4, 5]] == 9.0).all()
    c.n_q = [2, 1, 3]
    _check_rows(c, out, lse, [(1, 0)])


@pytest.mark.parametrize("amax", [1e-32, 1e30])
@pytest.mark.parametrize("lens", [[30, 1], [20000, 7]])
def test_values_of_any_magnitude(L, work, amax, lens):  # noqa: F811
    """Tensor scales near the ends of fp32's range, even weights over few and many keys, positive values (none cancels)."""
    from nvfp4_w4a4_quantized_quantize_gb300.kvcache import tensor_scale
    c = Case(lens, [1, 1], 8, 2, 128, 64, seed=7, q_scale=0.0)
    c.cache.v_codes &= 0x77
    c.cache.v_tscale.copy_(tensor_scale(amax))
    c.check(L, work)
