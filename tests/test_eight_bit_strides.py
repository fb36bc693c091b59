"""The 8-bit write refuses pages and scales whose heads, blocks or pages share a place (a stride of zero): their writers would race.
Reads of such pages are allowed.  On the host, before any launch (no GPU)."""
import ctypes

import pytest

from test_cache_refusals import _fake
from test_eight_bit_refusals import _eight


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


def _append(sd, a, pg, B=1):
    st = (ctypes.c_int64 * 3)(1024, 1024, 128)
    return sd.load_library().specdec_append_kv8(a, st, a, st, sd.BF16, a, None, B, 1, pg, None, None)


@pytest.mark.parametrize("name", ["page_stride", "head_stride", "scale_page_stride", "scale_slot_stride", "scale_head_stride"])
def test_shared_places_are_not_written(sd, name):
    a, keep = _fake()
    assert _append(sd, a, _eight(sd, a, num_pages=3, **{name: 0})) == sd.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(num_pages=1, page_stride=0, scale_page_stride=0), dict(kv_heads=1, head_stride=0, scale_head_stride=0),
                                    dict(scale_block=64, scale_slot_stride=0)])
def test_a_stride_that_does_not_count_may_be_zero(sd, change):
    """(B = 70000 is refused by the check behind this one: nothing is launched.)"""
    a, keep = _fake()
    assert _append(sd, a, _eight(sd, a, **{"num_pages": 3, **change}), B=70000) == sd.ERR_UNSUPPORTED
