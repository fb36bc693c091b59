"""The cache calls refuse what they cannot run, on the host and before any launch (no GPU)."""
import ctypes
import math

import pytest


def _fake(n=4096):
    buf = (ctypes.c_byte * (n + 256))()
    return (ctypes.addressof(buf) + 255) // 256 * 256, buf


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


def _pages(sd, addr, **kw):
    from speculative_decoding_token_temperature_gb300.cache import _KvPages
    d = dict(k=addr, v=addr, block_table=addr, page_stride=16 * 8 * 256, slot_stride=8 * 256, head_stride=256,
             num_pages=4, page_size=16, max_pages=2, kv_heads=8, head_dim=128, format=sd.BF16, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return _KvPages(**d)


def _four(sd, addr, **kw):
    d = dict(page_stride=16 * 8 * 64, slot_stride=8 * 64, head_stride=64, scale_page_stride=16 * 64, scale_slot_stride=64,
             scale_head_stride=8, k_scales=addr, v_scales=addr, format=sd.KV4)
    d.update(kw)
    return _pages(sd, addr, **d)


BAD_PAGES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(block_table=None), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
    (dict(max_pages=-1), 1), (dict(kv_heads=0), 1), (dict(format=0), 1), (dict(format=2), 1),
    (dict(page_stride=8), 2), (dict(slot_stride=-16), 2), (dict(head_stride=24), 2),
    (dict(max_pages=1 << 20, page_size=1 << 12), 2),
]


def _attend(sd, a, pages, **kw):
    st = (ctypes.c_int64 * 3)(32 * 128, 32 * 128, 128)
    d = dict(q=a, st=st, dt=sd.BF16, lens=a, ql=None, mask=None, depth=None, B=1, n=1, hq=32, window=0, sinks=0,
             scale=1.0, out=a, lse=None, status=None, ws=a, wsb=1 << 30)
    d.update(kw)
    return sd.load_library().specdec_attend(d["q"], d["st"], d["dt"], pages, d["lens"], d["ql"], d["mask"], d["depth"],
                                            d["B"], d["n"], d["hq"], d["window"], d["sinks"], d["scale"], d["out"],
                                            d["lse"], d["status"], d["ws"], d["wsb"], None)


@pytest.mark.parametrize("change,code", BAD_PAGES + [(dict(head_dim=96), 2), (dict(kv_heads=5), 1)])
def test_attend_refuses_bad_pages(sd, change, code):
    a, keep = _fake()
    assert _attend(sd, a, _pages(sd, a, **change)) == code


@pytest.mark.parametrize("change,code", [(dict(k_scales=None), 1), (dict(k_scale=0.0), 1), (dict(v_scale=math.inf), 1),
                                         (dict(k_scale=math.nan), 1), (dict(scale_slot_stride=12), 2),
                                         (dict(scale_head_stride=-8), 2)])
def test_four_bit_pages_are_checked(sd, change, code):
    a, keep = _fake()
    lib = sd.load_library()
    pg = _four(sd, a, **change)
    st = (ctypes.c_int64 * 3)(1024, 1024, 128)
    assert _attend(sd, a, pg) == code
    assert lib.specdec_append_kv4(a, st, a, st, sd.BF16, a, None, 1, 1, pg, None, None) == code
    assert lib.specdec_read_kv4(a, None, 1, 1, pg, sd.F16, a, a, None, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(st=None), 1), (dict(dt=0), 1), (dict(dt=3), 1), (dict(B=0), 1), (dict(n=0), 1), (dict(hq=0), 1),
    (dict(window=-1), 1), (dict(sinks=-2), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(ws=None), 1), (dict(wsb=16), 4), (dict(hq=12), 1), (dict(n=1 << 23), 2), (dict(hq=8 << 16), 2),
    (dict(st=(ctypes.c_int64 * 3)(4, 8, 8)), 2), (dict(st=(ctypes.c_int64 * 3)(8, -8, 8)), 2),
])
def test_attend_refuses_bad_arguments(sd, change, code):
    a, keep = _fake()
    assert _attend(sd, a, _pages(sd, a), **change) == code


def test_attend_refuses_misaligned_and_mismatched(sd):
    a, keep = _fake()
    assert _attend(sd, a, None) == 1
    assert _attend(sd, a, _pages(sd, a), q=a + 2) == 2
    assert _attend(sd, a, _pages(sd, a), out=a + 4) == 2
    assert _attend(sd, a, _pages(sd, a), ws=a + 16) == 1
    assert _attend(sd, a, _pages(sd, a), depth=a) == 1
    assert _attend(sd, a, _pages(sd, a, k=a + 8)) == 2
    assert sd.load_library().specdec_attend_workspace_bytes(1, 1, 32, 8, 128) > 0
    for bad in ((0, 1, 32, 8, 128), (1, 0, 32, 8, 128), (1, 1, 32, 5, 128), (1, 1, 32, 8, 96)):
        assert sd.load_library().specdec_attend_workspace_bytes(*bad) == 0


def _rotate(sd, a, **kw):
    st = (ctypes.c_int64 * 3)(6144, 6144, 128)
    d = dict(q=a, qs=st, k=a, ks=st, v=a, vs=st, dt=sd.BF16, qw=None, kw=None, eps=1e-6, turns=a, rot=128, il=0, lens=a,
             ql=None, depth=None, B=1, n=1, hq=32, hkv=8, D=128, oq=a, ok=None, pages=_pages(sd, a), status=None)
    d.update(kw)
    return sd.load_library().specdec_rotate_qk(*(d[x] for x in (
        "q", "qs", "k", "ks", "v", "vs", "dt", "qw", "kw", "eps", "turns", "rot", "il", "lens", "ql", "depth", "B", "n",
        "hq", "hkv", "D", "oq", "ok", "pages", "status")), None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(vs=None), 1), (dict(dt=0), 1), (dict(B=0), 1), (dict(n=0), 1),
    (dict(hq=0), 1), (dict(hkv=4), 1), (dict(D=96, rot=96), 2), (dict(rot=0), 1), (dict(rot=130), 1), (dict(rot=24), 2),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(turns=None), 1), (dict(lens=None), 1), (dict(oq=None), 1),
    (dict(pages=None), 1), (dict(B=70000), 2), (dict(D=64, rot=64), 1),
])
def test_rotate_refuses_bad_arguments(sd, change, code):
    a, keep = _fake()
    assert _rotate(sd, a, **change) == code


def test_rotate_takes_pages_or_an_output_not_both(sd):
    a, keep = _fake()
    assert _rotate(sd, a, ok=a) == 1
    assert _rotate(sd, a, q=a + 8) == 2
    assert _rotate(sd, a, qw=a + 2) == 2
    assert _rotate(sd, a, pages=_four(sd, a)) == 1


@pytest.mark.parametrize("change,code", [(dict(dt=0), 1), (dict(B=0), 1), (dict(n=0), 1), (dict(lens=None), 1),
                                         (dict(B=70000), 2), (dict(n=1 << 24), 2), (dict(k=None), 1)])
def test_append_and_read_refuse_bad_arguments(sd, change, code):
    a, keep = _fake()
    st = (ctypes.c_int64 * 3)(1024, 1024, 128)
    d = dict(k=a, dt=sd.BF16, lens=a, B=1, n=1)
    d.update(change)
    lib = sd.load_library()
    assert lib.specdec_append_kv4(d["k"], st, a, st, d["dt"], d["lens"], None, d["B"], d["n"], _four(sd, a), None, None) == code
    assert lib.specdec_read_kv4(d["lens"], None, d["B"], d["n"], _four(sd, a), d["dt"], d["k"], a, None, None) == code
    assert lib.specdec_append_kv4(a, st, a, st, sd.BF16, a, None, 1, 1, _pages(sd, a), None, None) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes(sd):
    import torch
    q = torch.zeros(1, 1, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(2, 16, 8, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for call in (lambda: sd.attend(q, pool, pool, table, lens),
                 lambda: sd.rotate_qk(q, q, torch.zeros(64, dtype=torch.int64), lens),
                 lambda: sd.append_kv4(q, q, pool, pool, table, lens, k_scales=None, v_scales=None),
                 lambda: sd.read_kv4(pool, pool, table, lens, 1, k_scales=None, v_scales=None),
                 lambda: sd.attend(q.float(), pool, pool, table, lens),
                 lambda: sd.attend(q[0], pool, pool, table, lens)):
        with pytest.raises(ValueError):
            call()


def test_rotation_turns_are_exact_counts(sd):
    t = sd.rotation_turns([2 * math.pi * 0.25, 2 * math.pi * 0.75, 2 * math.pi * 1.25, 0.0])
    assert t.tolist() == [1 << 62, -(1 << 62), 1 << 62, 0]


def test_kernel_hook_values(sd):
    assert sd.load_library().specdec_set_test_hook(sd.HOOK_ATTEND_KERNEL, 3) == sd.ERR_INVALID_ARG
    with sd.test_hooks(attend_kernel=2):
        assert sd.get_test_hook(sd.HOOK_ATTEND_KERNEL) == 2
    assert sd.get_test_hook(sd.HOOK_ATTEND_KERNEL) == 0
