"""Limits of the decode step's entries that follow from sizes taken together, and alignments of every pointer, on the
CPU: refused on the host before any CUDA call.  The pointers are placeholders that are never read."""
import pytest

from tests.test_decode_errors import ALIGN, LIB, P, SHAPE, _attend, _cache, _refused


@pytest.mark.parametrize("kw", [
    dict(heads=65534, max_q=65535), dict(heads=16386, max_q=65535),
    dict(heads=8192, max_q=65535, B=1 << 20, blocks=1 << 26, ld=1 << 26), dict(heads=1024, max_q=65535, B=1 << 20, blocks=1 << 16, ld=1 << 16)])
def test_attention_refuses_work_that_its_units_cannot_count(kw):
    _refused(_attend(_cache(), q_off=P, rows=1 << 20, **kw), SHAPE, "nvfp4_kv_attention")


@pytest.mark.parametrize("name", ["new", "len", "table", "free", "count", "len_out", "count_out", "q_off", "slots", "pos"])
def test_plan_refuses_every_pointer_off_its_elements(name):
    """The kernel reads and writes whole elements: an odd address would fault."""
    a = {n: P + 4096 * i for i, n in enumerate(["new", "len", "table", "free", "count", "len_out", "count_out", "q_off", "slots", "pos"])}
    a[name] += 2
    _refused(LIB.nvfp4_kv_plan(a["new"], a["len"], 4, 16, a["table"], 4, 4, a["free"], 8, a["count"], a["len_out"], a["count_out"],
                               a["q_off"], a["slots"], a["pos"], 64, None), ALIGN, "nvfp4_kv_plan")
