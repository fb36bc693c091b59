"""The calls on 8-bit pages refuse what they cannot run, on the host and before any launch (no GPU)."""
import ctypes
import math

import pytest

from test_cache_refusals import _attend, _fake, _pages


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


def _eight(sd, addr, **kw):
    d = dict(page_size=64, page_stride=64 * 8 * 128, slot_stride=8 * 128, head_stride=128, scale_page_stride=2 * 8, scale_slot_stride=8,
             scale_head_stride=1, k_scales=addr, v_scales=addr, format=sd.KV8, scale_block=32)
    d.update(kw)
    return _pages(sd, addr, **d)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), 1), (dict(v_scales=None), 1), (dict(k_scales=None), 1), (dict(block_table=None), 1), (dict(num_pages=0), 1),
    (dict(k_scale=0.0), 1), (dict(v_scale=math.inf), 1), (dict(k_scale=math.nan), 1), (dict(v_scale=-1.0), 1), (dict(k_scale=1e-40), 1),
    (dict(scale_block=0), 1), (dict(scale_block=-16), 1), (dict(scale_block=8), 2), (dict(scale_block=48), 2), (dict(scale_block=128), 2),
    (dict(page_size=24, scale_block=16), 2), (dict(scale_page_stride=-1), 2), (dict(scale_slot_stride=-8), 2), (dict(scale_head_stride=-1), 2),
    (dict(slot_stride=1000), 2), (dict(page_stride=-16), 2), (dict(head_dim=96), 2), (dict(max_pages=1 << 20, page_size=1 << 12), 2),
    (dict(format=5), 1),
])
def test_eight_bit_pages_are_checked(sd, change, code):
    a, keep = _fake()
    lib = sd.load_library()
    pg = _eight(sd, a, **change)
    st = (ctypes.c_int64 * 3)(1024, 1024, 128)
    assert _attend(sd, a, pg) == code
    assert lib.specdec_append_kv8(a, st, a, st, sd.BF16, a, None, 1, 1, pg, None, None) == code
    assert lib.specdec_read_kv8(a, None, 1, 1, pg, sd.F16, a, a, None, None) == code


@pytest.mark.parametrize("change,code", [(dict(dt=0), 1), (dict(dt=4), 1), (dict(B=0), 1), (dict(n=0), 1), (dict(lens=None), 1),
                                         (dict(B=70000), 2), (dict(n=1 << 24), 2), (dict(k=None), 1)])
def test_append_and_read_refuse_bad_arguments(sd, change, code):
    a, keep = _fake()
    st = (ctypes.c_int64 * 3)(1024, 1024, 128)
    d = dict(k=a, dt=sd.BF16, lens=a, B=1, n=1)
    d.update(change)
    lib = sd.load_library()
    assert lib.specdec_append_kv8(d["k"], st, a, st, d["dt"], d["lens"], None, d["B"], d["n"], _eight(sd, a), None, None) == code
    assert lib.specdec_read_kv8(d["lens"], None, d["B"], d["n"], _eight(sd, a), d["dt"], d["k"], a, None, None) == code


def test_formats_are_not_mixed(sd):
    a, keep = _fake()
    lib = sd.load_library()
    st = (ctypes.c_int64 * 3)(1024, 1024, 128)
    four = _eight(sd, a, format=sd.KV4)
    for pg in (_pages(sd, a), four, None):
        assert lib.specdec_append_kv8(a, st, a, st, sd.BF16, a, None, 1, 1, pg, None, None) == 1
        assert lib.specdec_read_kv8(a, None, 1, 1, pg, sd.F16, a, a, None, None) == 1
    eight = _eight(sd, a)
    assert lib.specdec_append_kv4(a, st, a, st, sd.BF16, a, None, 1, 1, eight, None, None) == 1
    assert lib.specdec_read_kv4(a, None, 1, 1, eight, sd.F16, a, a, None, None) == 1
    odd = (ctypes.c_int64 * 3)(1020, 1024, 128)
    assert lib.specdec_append_kv8(a, odd, a, st, sd.BF16, a, None, 1, 1, eight, None, None) == 2
    assert lib.specdec_append_kv8(a + 8, st, a, st, sd.BF16, a, None, 1, 1, eight, None, None) == 2
    assert lib.specdec_read_kv8(a, None, 1, 1, eight, sd.F16, a + 8, a, None, None) == 2


def test_binding_refuses_host_tensors_and_wrong_shapes(sd):
    import torch
    q = torch.zeros(1, 1, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(2, 32, 8, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros(2, 2, 8, dtype=torch.uint8)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    kw = dict(k_scales=scales, v_scales=scales)
    for call in (lambda: sd.attend(q, pool, pool, table, lens, **kw),
                 lambda: sd.append_kv8(q, q, pool, pool, table, lens, **kw),
                 lambda: sd.append_kv8(q.float(), q, pool, pool, table, lens, **kw),
                 lambda: sd.read_kv8(pool, pool, table, lens, 1, **kw),
                 lambda: sd.read_kv8(pool, pool, table, lens, 1, dtype=torch.float32, **kw)):
        with pytest.raises(ValueError):
            call()
