"""Limits of the decode step's entries that follow from sizes taken together, and alignments of every pointer, on the
CPU: refused on the host before any CUDA call.  The pointers are placeholders that are never read."""
import pytest

from tests.test_decode_errors import P, SHAPE, _attend, _cache, _refused


@pytest.mark.parametrize("kw", [
    dict(heads=65534, max_q=65535), dict(heads=16386, max_q=65535),
    dict(heads=8192, max_q=65535, B=1 << 20, blocks=1 << 26, ld=1 << 26), dict(heads=1024, max_q=65535, B=1 << 20, blocks=1 << 16, ld=1 << 16)])
def test_attention_refuses_work_that_its_units_cannot_count(kw):
    _refused(_attend(_cache(), q_off=P, rows=1 << 20, **kw), SHAPE, "nvfp4_kv_attention")
