"""The cache calls at the edges of their contracts: values that are not finite, scales and weights
next to 0, the widest windows, arguments without a truth value, workspaces.

Tolerances are those of test_gpu_cache.py unless a test derives its own.
"""
import numpy as np
import pytest
import torch

import test_gpu_cache as base
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


@pytest.fixture(params=["rule", "warp", "tensor_memory"])
def kernel(request, hooks):
    """Each case through the kernel that the rule picks, and through each kernel."""
    hooks(attend_kernel=("rule", "warp", "tensor_memory").index(request.param))
    return request.param


def _same_places(r, c, q, lens, dtype, D, **mask):
    """Finite outputs as the oracle's, and the others at the oracle's places (an infinity may come out as NaN:
    0 times it is)."""
    for b, L in enumerate(lens):
        n = q.shape[1]
        k, v = c.rows(b, L)
        out, lse, pv, av, qk = co.attend(base._np(q[b]), k, v, co.visible(n, n, L, mask.get("window", 0), mask.get("sinks", 0)), D ** -0.5)
        odd = ~np.isfinite(out)
        got = r["out"][b].clone()
        assert np.array_equal(~np.isfinite(base._np(got)), odd), (b, np.argwhere(~np.isfinite(base._np(got)) != odd)[:4])
        got[torch.tensor(odd, device=DEV)] = 0
        out[odd] = pv[odd] = av[odd] = 0
        base._check(got, r["lse"][b], (out, lse, pv, av, qk), dtype, c.four, D, f"b={b}")


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("n", [33, 64, 300])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 0), (70, 3), (600, 20)])
def test_odd_values_under_two_row_tiles(sd, four, D, dtype, n, window, sinks):
    """More than 128 query rows to a key head: two row tiles share the staged values, and a tile of slots may
    be whole for one and partial for the other.  Every request holds one such value: seen by all rows, by the
    later ones, by the earlier ones (a window's low edge), or as one of the first slots."""
    first = [100, 100, 127, 250, 5, 640, 400, 700]
    slots = [5, 104, 127 + n // 2, 130, 0, 640 + n - 2, 400 + n // 2 - 140, 2]
    lens = [p + n for p in first]
    c = base.Cache(len(lens), max(lens), 16, 1, D, dtype, four)
    for b, s in enumerate(slots):
        if four:
            c.vs[int(c.host_table[b, s // 16]), s % 16, :, b % (D // 16)] = 0x7f
        else:
            c.put("v", b, s, float("inf") if b % 3 == 1 else float("nan"))
    q = base._q(len(lens), n, 4, D, dtype)
    for _ in range(3):
        r = sd.attend(q, c.k, c.v, c.table, base._i32(lens), window=window, sinks=sinks, with_lse=True, **c.kw)
        torch.cuda.synchronize()
        assert not r["status"].any()
        _same_places(r, c, q, lens, dtype, D, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 7, 20, 40])
@pytest.mark.parametrize("scale", [0.0, 1e-44, -1e-44, 1e-38])
def test_scales_next_to_zero_over_four_bit_pages(sd, kernel, D, n, scale):
    """bf16 queries below 1, whose rows carry a power of two below 1 of their own: its product with the scale
    may vanish, and masked slots stay masked."""
    c = base.Cache(2, 300, 16, 1, D, BF16, True)
    base._run(sd, c, base._q(2, n, 4, D, BF16, std=0.1), [n, 299], BF16, D, scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 7, 20, 40])
def test_scores_of_minus_infinity(sd, kernel, dtype, n):
    """A visible score of -inf among finite ones has the weight 0; where all of a row's are -inf (or one is
    +inf) the softmax has no value, and the row is NaN."""
    D, page = 64, 16
    lens = [n + 200, n + 5, n + 150]
    c = base.Cache(3, max(lens), page, 1, D, dtype)
    q = base._q(3, n, 4, D, dtype).abs() + 0.5

    def key(b, slot, value):
        c.k[int(c.host_table[b, slot // page]), slot % page, :, 3] = value

    low = {0: [5, 130, lens[0] - 1], 1: list(range(6)), 2: []}
    for b, slots in low.items():
        for s in slots:
            key(b, s, float("-inf"))
    key(2, lens[2] - 1, float("inf"))
    r = sd.attend(q, c.k, c.v, c.table, base._i32(lens), with_lse=True)
    torch.cuda.synchronize()
    assert not r["status"].any()
    for b, L in enumerate(lens):
        sees = co.visible(n, n, L, 0, 0)
        sees[:, low[b]] = False  # what is left of the softmax
        some = sees.any(1)
        if b == 2:
            some = some & ~sees[:, L - 1]
        k, v = c.rows(b, L)
        want = co.attend(base._np(q[b, some]), k, v, sees[some], D ** -0.5)
        base._check(r["out"][b, some], r["lse"][b, some], want, dtype, False, D, f"b={b}")
        assert torch.isnan(r["out"][b, ~some]).all() and torch.isnan(r["lse"][b, ~some]).all(), b
        assert b == 0 or not some.all()


def test_all_scores_of_minus_infinity_in_parts_and_beside_empty_rows(sd, kernel):
    D = 128
    c = base.Cache(1, 5000, 64, 1, D, BF16)
    c.k[..., 0] = float("-inf")
    q = base._q(1, 1, 2, D, BF16).abs() + 0.5
    r = sd.attend(q, c.k, c.v, c.table, base._i32([5000]), with_lse=True)  # parts of many CTAs
    torch.cuda.synchronize()
    assert torch.isnan(r["out"]).all() and torch.isnan(r["lse"]).all()
    # a tree's rows that see no slot stay zeros: by the mask, or for a sequence that is shorter
    n = 5
    mask = np.tril(np.ones((n, n), np.uint8))
    mask[1] = 0
    q = base._q(1, n, 2, D, BF16).abs() + 0.5
    kw = dict(query_len=base._i32([4]), tree_mask=torch.tensor(mask, device=DEV), with_lse=True)
    depth = dict(depth=base._i32([0, 1, 1, 2, 2]))
    for extra, first, empty in (({}, 0, (1, 4)), ({}, 3, (4,)), (dict(window=1, **depth), 3, (1, 4)), (dict(window=2), 3, (1, 4)),
                                (dict(window=2, sinks=1), 3, (4,))):
        r = sd.attend(q, c.k, c.v, c.table, base._i32([first + 4]), **kw, **extra)
        torch.cuda.synchronize()
        for i in range(n):
            if i in empty:
                assert not r["out"][0, i].any() and torch.isneginf(r["lse"][0, i]).all(), (extra, first, i)
            else:
                assert torch.isnan(r["out"][0, i]).all() and torch.isnan(r["lse"][0, i]).all(), (extra, first, i)


@pytest.mark.parametrize("dtype,four", [(F16, False), (F16, True), (BF16, True)])
@pytest.mark.parametrize("n,hq", [(1, 2), (4, 4), (12, 4), (40, 4)])
def test_many_small_weights_beside_a_large_one(sd, kernel, dtype, four, n, hq):
    """A first slot 26 bits above 2000 equal ones, its value 0: the output is theirs alone.  A weight is
    rounded in fp16 relative to a reference of 2^7 or more, so to 2^-25 2^-7 of the row's largest.
    (160 requests share the pages, so that an item's tiles stay on a CTA.)"""
    D, B = 64, 160
    L = 2000 + n
    c = base.Cache(1, L, 16, 1, D, dtype, four)
    k = torch.zeros(1, L, 1, D, dtype=dtype, device=DEV)
    k[0, 0, 0, 0] = 12.0
    v = (30 + base._q(1, L, 1, D, dtype)).contiguous()
    v[0, 0] = 0
    if four:
        c.kw.update(k_scale=1.0, v_scale=1.0)
        sd.append_kv4(k, v, c.k, c.v, c.table, base._i32([L]), **c.kw)
    else:
        at = torch.arange(L)
        c.k[c.host_table[0].long()[at // 16].to(DEV), (at % 16).to(DEV)] = k[0]
        c.v[c.host_table[0].long()[at // 16].to(DEV), (at % 16).to(DEV)] = v[0]
    q = torch.zeros(B, n, hq, D, dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    scale = 26 * np.log(2) / 12
    r = sd.attend(q, c.k, c.v, c.table.expand(B, -1).contiguous(), base._i32([L] * B), scale=scale, with_lse=True, **c.kw)
    torch.cuda.synchronize()
    keys, values = c.rows(0, L)
    out, lse, pv, av, qk = co.attend(base._np(q[0]), keys, values, co.visible(n, n, L, 0, 0), scale)
    es = D * 2.0 ** -24 * qk
    tol = ((2 * es + 2.0 ** -13)[..., None] + base.U[F16]) * pv + 2.0 ** -32 * av + base.U[dtype] * np.abs(out) + 2.0 ** -25
    assert (np.abs(base._np(r["out"]) - out) <= tol).all(), (np.abs(base._np(r["out"]) - out).max(), tol.min())
    assert (np.abs(base._np(r["lse"]) - lse) <= es + 2.0 ** -13 + 2.0 ** -22 * np.abs(lse)).all()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 30, 2 ** 30])
@pytest.mark.parametrize("hq", [1, 4])
def test_windows_beyond_every_position(sd, kernel, window, hq):
    """New tokens that all see each other, under a window as wide as an int goes."""
    n, D = 40, 64
    c = base.Cache(3, 240, 16, 1, D, F16)
    q = base._q(3, n, hq, D, F16)
    base._run(sd, c, q, [n, n + 30, n + 200], F16, D, mask=np.ones((n, n), np.uint8), window=window, sinks=2)
    base._run(sd, c, q, [n, n + 30, n + 200], F16, D, window=window)


@pytest.mark.parametrize("page", [1, 5])
@pytest.mark.parametrize("window,sinks", [(3, 0), (21, 2)])
def test_entries_behind_the_window_within_a_step(sd, kernel, page, window, sinks):
    """Pages out of range between the first slots and the window, in the same 16 slots as visible ones."""
    D, L, n = 64, 75, 2
    c = base.Cache(1, L, page, 2, D, BF16)
    for p in range(c.table.shape[1]):
        if p * page >= sinks and (p + 1) * page <= L - n - (window - 1):
            c.table[0, p] = -5 if p % 2 else 1 << 30
    base._run(sd, c, base._q(1, n, 4, D, BF16), [L], BF16, D, window=window, sinks=sinks)


def test_flags_without_a_truth_value_raise_their_error(sd):
    c = base.Cache(1, 16, 16, 1, 64, BF16)
    q, k = base._q(1, 1, 2, 64, BF16), base._q(1, 1, 1, 64, BF16)
    many = torch.ones(2, dtype=torch.bool)
    for call in (lambda: sd.attend(q, c.k, c.v, c.table, base._i32([3]), with_lse=many),
                 lambda: sd.rotate_qk(q, k, sd.rotation_turns([1.0] * 32, DEV), base._i32([3]), interleaved=many)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()
    torch.cuda.synchronize()


def test_workspaces_of_many_streams_are_let_go(sd):
    """The workspaces that calls leave do not grow with the streams they ran on."""
    c = base.Cache(2, 400, 16, 1, 128, F16)
    q, lens = base._q(2, 300, 1, 128, F16), base._i32([400, 390])
    want = sd.attend(q, c.k, c.v, c.table, lens)["out"]
    torch.cuda.synchronize()
    held = []
    streams = [torch.cuda.Stream() for _ in range(24)]
    for s in streams:
        r = sd.attend(q, c.k, c.v, c.table, lens, stream=s)
        s.synchronize()
        assert torch.equal(r["out"], want)
        del r
        held.append(torch.cuda.memory_allocated())
    assert len({s.cuda_stream for s in streams}) == 24 and held[11] == held[23]
    # one stream after another, without a wait: what is let go may still be in use
    got = [sd.attend(q, c.k, c.v, c.table, lens, stream=s)["out"] for s in streams + streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
