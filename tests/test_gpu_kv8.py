"""GPU parity of the calls on 8-bit pages (the write, the read, attention) against the fp64 oracle, at the sizes, masks,
strides and contents where they can go wrong.

Tolerances.  Codes and scales: exact.  Values read back: one rounding.  Attention: as over 4-bit pages
(test_gpu_cache.py), for the staged values are exact in fp16 as those are: weights of fp16, fp32 sums, one rounding at the end.
"""
import numpy as np
import pytest
import torch

import test_gpu_cache as base
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F16 = torch.bfloat16, torch.float16
LEAST, MOST = -15, 7


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


class Cache(base.Cache):
    """8-bit pages of B sequences in a shuffled order; layout "views": inside wider tensors, heads outermost."""

    def __init__(self, B, max_len, page, block, hkv, D, seed=0, layout="plain", std=100.0, exps=(-8, -3)):
        g = torch.Generator().manual_seed(seed)
        per = max(1, -(-max_len // page))
        self.N, self.page, self.block, self.four = B * per + 3, page, block, True
        self.host_table = torch.randperm(self.N, generator=g)[:B * per].view(B, per).to(torch.int32)
        self.table = self.host_table.to(DEV)
        N, blocks = self.N, page // block

        def codes():
            x = (torch.randn(N, page, hkv, D, generator=g) * std).clamp(-448, 448).to(torch.float8_e4m3fn).to(DEV)
            if layout == "plain":
                return x
            wide = torch.zeros(N, hkv + 1, page, D + 16, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
            view = wide[:, 1:, :, :D].permute(0, 2, 1, 3)
            view.view(torch.uint8).copy_(x.view(torch.uint8))
            return view

        def scales():
            x = torch.randint(127 + exps[0], 127 + exps[1] + 1, (N, blocks, hkv), generator=g, dtype=torch.uint8).to(DEV)
            if layout == "plain":
                return x
            wide = torch.zeros(N, hkv, blocks + 3, dtype=torch.uint8, device=DEV)
            view = wide[:, :, 1:blocks + 1].permute(0, 2, 1)
            view.copy_(x)
            return view.view(torch.float8_e8m0fnu)

        self.k, self.v, self.ks, self.vs = codes(), codes(), scales(), scales()
        self.kw = dict(k_scales=self.ks, v_scales=self.vs, k_scale=0.375, v_scale=1.5)

    def where(self, b, L):
        s = torch.arange(L)
        return self.host_table[b].long()[s // self.page].to(DEV), (s % self.page).to(DEV)

    def exps(self, which, b, L):
        """Exponents of sequence b's first L slots [L, Hkv]."""
        pg, off = self.where(b, L)
        return getattr(self, which + "s").view(torch.uint8)[pg, off // self.block].cpu().numpy().astype(int) - 127

    def codes(self, which, b, L):
        pg, off = self.where(b, L)
        return getattr(self, which).view(torch.uint8)[pg, off].cpu().numpy()

    def rows(self, b, L):
        return tuple(co.decode8(self.codes(w, b, L), self.exps(w, b, L)[..., None]) * np.float32(self.kw[w + "_scale"]) for w in "kv")

    def put(self, which, b, slot, value):
        getattr(self, which).view(torch.uint8)[int(self.host_table[b, slot // self.page]), slot % self.page] = value


def _new(B, n, hkv, D, dtype, seed=3, std=1.0, spread=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, n, hkv, D, generator=g) * std
    if spread:
        x = x * 2.0 ** torch.randint(-spread, spread + 1, (B, 1, hkv, 1), generator=g)
    return x.to(dtype).to(DEV)


def _append_and_check(sd, c, k, v, lens, nq=None, **kw):
    """The call against the oracle, bit for bit, everything it must not touch included; then the values read back."""
    B, n, hkv, D = k.shape
    nq = [n] * B if nq is None else nq
    old = {w: getattr(c, w).view(torch.uint8).clone() for w in ("k", "v", "ks", "vs")}
    want = {w: t.cpu().numpy().copy() for w, t in old.items()}
    for b, L in enumerate(lens):
        if nq[b] == 0:
            continue
        blocks = -(-L // c.block)
        for w, x in (("k", k), ("v", v)):
            for h in range(hkv):
                pages = c.host_table[b].numpy()
                slots = np.arange(blocks * c.block)
                pg, off = pages[slots // c.page], slots % c.page
                bp, bo = pages[np.arange(blocks) * c.block // c.page], np.arange(blocks) * c.block % c.page // c.block
                codes, exps = co.append8(want[w][pg, off, h], want[w + "s"][bp, bo, h].astype(int) - 127, base._np(x[b, :nq[b], h]), L - nq[b],
                                         c.block, c.kw[w + "_scale"])
                want[w][pg, off, h], want[w + "s"][bp, bo, h] = codes, exps + 127
    r = sd.append_kv8(k, v, c.k, c.v, c.table, base._i32(lens), query_len=base._i32(nq), **c.kw, **kw)
    torch.cuda.synchronize()
    assert not r["status"].any()
    for w in ("ks", "vs", "k", "v"):
        got = getattr(c, w).view(torch.uint8).cpu().numpy()
        differ = np.argwhere((got != want[w]) & ~((w in "kv") & ((got & 127) == 127) & ((want[w] & 127) == 127)))
        assert len(differ) == 0, (w, differ[:5], [(got[tuple(i)], want[w][tuple(i)]) for i in differ[:5]])
    dtype = k.dtype
    r = sd.read_kv8(c.k, c.v, c.table, base._i32(lens), n, query_len=base._i32(nq), dtype=dtype, **c.kw)
    torch.cuda.synchronize()
    assert not r["status"].any()
    for b, L in enumerate(lens):
        rows = c.rows(b, L)
        for w, x in zip("kv", rows):
            got = base._np(r[w][b])
            x = x[L - nq[b]:]
            assert not got[nq[b]:].any()
            with np.errstate(invalid="ignore"):
                ok = (np.abs(got[:nq[b]] - x) <= base.U[dtype] * np.abs(x) + 2.0 ** -25) | (np.isnan(got[:nq[b]]) & np.isnan(x))
            assert ok.all()


# ---- the write ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page,block,hkv,D", [(16, 16, 1, 64), (64, 64, 2, 128), (96, 48, 3, 64), (256, 256, 1, 128), (1024, 512, 1, 64), (32, 16, 5, 128)])
@pytest.mark.parametrize("n", [1, 2, 8, 17, 70, 600])
def test_append_and_read(sd, dtype, page, block, hkv, D, n):
    lens = [n, n + 1, n + 15, n + block - 1, n + block, n + 5 + page]
    c = Cache(len(lens), max(lens), page, block, hkv, D, seed=n)
    _append_and_check(sd, c, _new(len(lens), n, hkv, D, dtype, spread=5), _new(len(lens), n, hkv, D, dtype, seed=4, spread=3), lens)


def test_rounds_of_appends_with_rejections(sd):
    """A cache that grows by rounds, some of whose tokens are rejected and written over: blocks' scales grow, and
    what was there follows."""
    B, hkv, D, block = 3, 2, 64, 32
    c = Cache(B, 200, 64, block, hkv, D)
    lens = [1, 30, 60]
    rng = np.random.default_rng(0)
    for step in range(12):
        n = 5
        lens = [L + n for L in lens]
        std = float(2.0 ** rng.integers(-4, 5))
        _append_and_check(sd, c, _new(B, n, hkv, D, BF16, seed=step, std=std), _new(B, n, hkv, D, BF16, seed=50 + step, std=std), lens)
        lens = [L - int(rng.integers(0, n)) for L in lens]  # rejected drafts


def test_values_at_the_ends_of_the_range(sd):
    """Zeros, values below and above the scales' range, infinities and NaN, and ties."""
    B, n, hkv, D = 1, 33, 2, 64
    c = Cache(B, 100, 16, 16, hkv, D)
    for dtype in (BF16, F16):
        for fill in (0.0, 2.0 ** -20, 1e-7, 60000.0, 3e4, 448.0 * 0.375, 452.0 * 0.375):
            k = torch.full((B, n, hkv, D), fill, dtype=dtype, device=DEV)
            k[0, ::2] *= -1
            k[0, 3, 0, 5], k[0, 4, 1, :] = float("nan"), float("inf")
            k[0, 32, :, 7] = float("-inf")
            _append_and_check(sd, c, k, k * 0.5, [n + 9])
    k = (torch.arange(n * D, device=DEV).view(1, n, 1, D).expand(1, n, hkv, D) % 512 - 256).to(BF16) * 0.375  # halfway values among them
    _append_and_check(sd, c, k.contiguous(), k.contiguous(), [n + 2])
    c.kw.update(k_scale=1e-36, v_scale=1e36)  # the product with 1 / k_scale overflows: saturated
    _append_and_check(sd, c, _new(B, n, hkv, D, BF16), _new(B, n, hkv, D, BF16), [n + 2])


def test_strided_pages_and_inputs(sd):
    B, n, hkv, D = 3, 9, 2, 128
    c = Cache(B, 150, 48, 16, hkv, D, layout="views")
    wide = _new(B, n, 3 * hkv, D, F16)
    _append_and_check(sd, c, wide[:, :, :hkv], wide[:, :, 2 * hkv:], [9, 77, 150])
    turned = _new(B, hkv, n, D, BF16).transpose(1, 2)
    _append_and_check(sd, c, turned, turned, [10, 50, 149], nq=[9, 0, 4])


def test_lengths_and_pages_in_error_leave_the_pages_alone(sd):
    B, n, hkv, D = 7, 20, 1, 64
    c = Cache(B, 64, 16, 16, hkv, D)
    table = c.table.clone()
    table[4, 2], table[5, 3] = c.N, -1
    before = {w: getattr(c, w).view(torch.uint8).clone() for w in ("k", "v", "ks", "vs")}
    lens, nq = base._i32([-1, 70, 15, 40, 45, 64, 30]), base._i32([20, 20, 20, -2, 20, 20, 0])
    k = _new(B, n, hkv, D, BF16)
    r = sd.append_kv8(k, k, c.k, c.v, table, lens, query_len=nq, **c.kw)
    torch.cuda.synchronize()
    assert r["status"].tolist() == [32] * 6 + [0]
    for w, t in before.items():
        assert torch.equal(getattr(c, w).view(torch.uint8), t)
    r = sd.read_kv8(c.k, c.v, table, lens, n, query_len=nq, **c.kw)
    torch.cuda.synchronize()
    assert r["status"].tolist() == [32] * 6 + [0] and torch.isnan(r["k"][:6]).all() and torch.isnan(r["v"][:6]).all() and not r["k"][6].any()
    r = sd.attend(_new(B, n, 2, D, BF16), c.k, c.v, table, lens, query_len=nq, with_lse=True, **c.kw)
    torch.cuda.synchronize()
    assert r["status"].tolist() == [32] * 6 + [0] and torch.isnan(r["out"][:4]).all() and not r["out"][6].any()


def test_rows_of_scales_may_hold_anything_behind_the_last_token(sd):
    """A fresh block's scale byte of before does not count."""
    c = Cache(2, 64, 32, 32, 1, 64)
    c.ks.fill_(255)
    c.vs.fill_(0)
    k = _new(2, 3, 1, 64, F16)
    sd.append_kv8(k, k, c.k, c.v, c.table, base._i32([3, 35]), **c.kw)
    torch.cuda.synchronize()
    for b, blk in ((0, 0), (1, 1)):
        pg = int(c.host_table[b, blk])
        e = co.block_exponent(float((base._np(k[b]).astype(np.float32) * np.float32(1 / np.float32(0.375))).__abs__().max()))
        assert int(c.ks[pg, 0, 0]) == e + 127


# ---- attention ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,D,n", [(8, 8, 64, 1), (8, 2, 128, 1), (16, 2, 128, 2), (7, 1, 64, 3), (12, 3, 128, 8), (28, 4, 128, 5), (4, 1, 64, 33),
                                        (10, 2, 128, 13), (40, 2, 64, 7)])
def test_chain_over_ragged_lengths(sd, kernel, dtype, hq, hkv, D, n):
    lens = [n, n + 1, 15 + n, 16 + n, 17 + n, 127 + n, 128 + n, 129 + n, 400 + n]
    c = Cache(len(lens), max(lens), 48, 16, hkv, D, seed=n)
    base._run(sd, c, base._q(len(lens), n, hq, D, dtype), lens, dtype, D, scale=0.05)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,n", [(1, 8), (1, 9), (1, 16), (1, 17), (1, 32), (1, 33), (3, 43), (1, 129), (2, 128), (1, 257), (5, 77)])
def test_row_tiles(sd, kernel, D, hq, n):
    """Query rows of a key head at and around the row tiles' borders, over one tile of 128 slots, two and several."""
    lens = [n, n + 100, n + 128, n + 500]
    c = Cache(len(lens), max(lens), 64, 32, 1, D, seed=n)
    base._run(sd, c, base._q(len(lens), n, hq, D, F16), lens, F16, D, scale=0.05)


@pytest.mark.parametrize("page,block", [(16, 16), (48, 16), (48, 48), (80, 16), (512, 256), (512, 512)])
def test_pages_and_blocks(sd, kernel, page, block):
    lens = [1, 16, 17, 63, 65, 333]
    c = Cache(len(lens), max(lens), page, block, 2, 128, seed=page, exps=(-15, 0))
    base._run(sd, c, base._q(len(lens), 1, 8, 128, BF16), lens, BF16, 128, scale=0.02)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (5, 1), (16, 16), (17, 4), (100, 40), (100000, 7), (64, 200)])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_window_and_sinks(sd, kernel, window, sinks, n):
    lens = [n, n + 3, n + 30, n + 155, n + 300]
    c = Cache(len(lens), max(lens), 32, 16, 2, 64, seed=window)
    base._run(sd, c, base._q(len(lens), n, 6, 64, F16), lens, F16, 64, window=window, sinks=sinks, scale=0.05)


@pytest.mark.parametrize("n,window,sinks", [(5, 0, 0), (17, 0, 0), (64, 0, 0), (64, 6, 2), (30, 3, 0), (2, 1, 1)])
def test_tree_masks(sd, kernel, n, window, sinks):
    lens = [n, n + 1, n + 29, n + 200]
    mask, depth, _ = base._tree(n, n)
    c = Cache(len(lens), max(lens), 32, 32, 2, 128, seed=n)
    base._run(sd, c, base._q(len(lens), n, 8, 128, BF16), lens, BF16, 128, mask=mask, depth=depth, window=window, sinks=sinks, scale=0.05)


def test_rows_that_see_nothing_and_tokens_that_do_not_exist(sd, kernel):
    n, D = 6, 64
    mask = np.tril(np.ones((n, n), np.uint8))
    mask[0] = mask[4] = 0  # with no prefix these rows are empty
    lens, nq = [6, 4, 0, 9, 40], [6, 4, 0, 6, 0]
    c = Cache(5, 40, 16, 16, 2, D)
    r = base._run(sd, c, base._q(5, n, 4, D, BF16), lens, BF16, D, nq=nq, mask=mask, scale=0.05)
    assert not r["out"][0, 0].any() and torch.isneginf(r["lse"][0, 4]).all()
    assert not r["out"][2].any() and not r["out"][4].any() and not r["out"][1, 4:].any()


def test_strided_pages_and_queries(sd, kernel):
    lens, D = [5, 100, 260], 128
    c = Cache(3, 260, 64, 32, 4, D, layout="views")
    wide = base._q(3, 5, 8 + 8, D, BF16)
    base._run(sd, c, wide[:, :, 8:], lens, BF16, D, scale=0.05)  # queries inside a fused projection's output
    turned = base._q(3, 8, 5, D, BF16).transpose(1, 2)  # heads before tokens
    base._run(sd, c, turned, lens, BF16, D, scale=0.05)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 8, 24, 40])
def test_masked_slots_may_hold_anything(sd, kernel, dtype, n):
    """Codes of NaN and any scale bytes behind the window, past the length and in nodes that a row does not see stay
    out of its result; rows that do see such codes get what the formula gives."""
    D, window, sinks = 128, 40, 2
    lens = [n + 100, n + 7]
    c = Cache(2, max(lens) + 40, 16, 16, 2, D)
    for b, L in enumerate(lens):
        for s in list(range(sinks, L - n - window)) + list(range(L, L + 20)):
            c.put("k", b, s, 0x7f)
            c.put("v", b, s, 0xff if s % 2 else 0x7f)
        last = (L - 1) // 16 + 1  # blocks past the last token, and between the first ones and the window
        for blk in list(range(last, last + 2)) + list(range(1, (L - n - window) // 16)):
            for w in ("ks", "vs"):
                getattr(c, w)[int(c.host_table[b, blk])] = 255 if blk % 2 else 0
    base._run(sd, c, base._q(2, n, 8, D, dtype), lens, dtype, D, window=window, sinks=sinks, scale=0.05, what="outside")
    # a later draft's key and value are NaN: only the rows that see it are touched
    c.put("v", 0, lens[0] - 1, 0x7f)
    if n > 2:
        c.put("v", 0, lens[0] - 2, 0xff)
        c.put("k", 1, lens[1] - 2, 0x7f)
    r = base._run(sd, c, base._q(2, n, 8, D, dtype), lens, dtype, D, window=window, sinks=sinks, scale=0.05, what="inside")
    if n > 2:
        assert torch.isfinite(r["out"][0, :n - 2]).all() and torch.isnan(r["out"][0, n - 1]).all()


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("n", [33, 64, 300])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 0), (70, 3), (600, 20)])
def test_single_codes_of_nan(sd, kernel, D, dtype, n, window, sinks):
    """One code of NaN in each request: seen by all rows, by the later ones, by the earlier ones, or as a first slot;
    one value of the rows that see it is NaN, the others are not."""
    first = [100, 100, 127, 250, 5, 640, 400, 700]
    slots = [5, 104, 127 + n // 2, 130, 0, 640 + n - 2, 400 + n // 2 - 140, 2]
    lens = [p + n for p in first]
    c = Cache(len(lens), max(lens), 32, 32, 1, D)
    for b, s in enumerate(slots):
        c.v.view(torch.uint8)[int(c.host_table[b, s // 32]), s % 32, :, (7 * b) % D] = 0x7f
    q = base._q(len(lens), n, 4, D, dtype)
    for _ in range(2):
        base._run(sd, c, q, lens, dtype, D, window=window, sinks=sinks, scale=0.05)


def _run_small(sd, c, q, lens, dtype, D, scale):
    """base._run for outputs that are subnormal in fp16: below 2^-14 its numbers are 2^-24 apart, so that the last
    rounding is off by up to 2^-25 whatever the value, where the tolerance there counts 2^-11 of the value alone."""
    n = q.shape[1]
    r = sd.attend(q, c.k, c.v, c.table, base._i32(lens), scale=scale, with_lse=True, **c.kw)
    torch.cuda.synchronize()
    assert not r["status"].any()
    for b, L in enumerate(lens):
        k, v = c.rows(b, L)
        out, lse, pv, av, qk = co.attend(base._np(q[b]), k, v, co.visible(n, n, L, 0, 0), scale)
        es = D * 2.0 ** -24 * qk
        tol = ((2 * es + 2.0 ** -13)[..., None] + base.U[F16]) * pv + 2.0 ** -25 * av + base.U[dtype] * np.abs(out)
        tol += 2.0 ** -25 if dtype == F16 else 1e-30
        assert (np.abs(base._np(r["out"][b]) - out) <= tol).all(), (np.abs(base._np(r["out"][b]) - out).max(), tol.min())
        assert (np.abs(base._np(r["lse"][b]) - lse) <= es + 2.0 ** -13 + 2.0 ** -22 * np.abs(lse)).all()


def test_scales_at_the_ends_of_the_range(sd, kernel):
    """Blocks of 2^-15 beside blocks of 2^7, for keys and for values, and codes of every magnitude."""
    for dtype in (BF16, F16):
        c = Cache(2, 300, 16, 16, 1, 64, exps=(LEAST, MOST))
        base._run(sd, c, base._q(2, 3, 4, 64, dtype, std=1e-3), [40, 300], dtype, 64, scale=0.03)
        c = Cache(2, 300, 16, 16, 1, 64, exps=(MOST, MOST), std=1000.0)
        base._run(sd, c, base._q(2, 20, 4, 64, dtype, std=1e-4), [40, 300], dtype, 64, scale=0.03)
        c = Cache(2, 300, 16, 16, 1, 64, exps=(LEAST, LEAST), std=0.01)
        _run_small(sd, c, base._q(2, 3, 40, 64, dtype), [40, 300], dtype, 64, scale=0.03)
    c = Cache(2, 90, 16, 16, 1, 64)  # bf16 queries far beyond fp16's range, and far below it
    for std in (1e30, 1e-30, 0.0):
        base._run(sd, c, base._q(2, 2, 4, 64, BF16, std=std), [3, 90], BF16, 64, scale=0.0 if std == 0 else 0.01 / std, what=f"queries of {std}")


@pytest.mark.parametrize("n", [2, 7, 20, 40])
@pytest.mark.parametrize("scale", [0.0, 1e-44, -1e-44, 1e-38, -0.05])
def test_scales_next_to_zero_and_below(sd, kernel, n, scale):
    c = Cache(2, 300, 16, 16, 1, 128)
    base._run(sd, c, base._q(2, n, 4, 128, BF16, std=0.1), [n, 299], BF16, 128, scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [3, 8, 40])
def test_queries_with_a_few_large_values(sd, kernel, dtype, D, n):
    """Rows of a few values 2^10 times the others', and of values of every magnitude.  Where queries are held in E4M3 pieces a
    value is off by at most 2^-17 of the row's largest (the largest is scaled into [128, 256), and what the pieces leave is at most half
    the smallest code, 2^-10): a score by 2^-17 scale max|q| sum|k| more, which counts like its other errors, twice for an
    output.  (1 + d for e^d is off by less than d^2, here below d / 32: 2.0625 instead of 2.)"""
    B, hq, hkv, scale = 2, 8, 2, 2.0 ** -13
    c = Cache(B, 300, 32, 16, hkv, D, seed=n)
    q = base._q(B, n, hq, D, F16 if dtype == F16 else torch.float32)
    q = q.float() * 2.0 ** -6
    q[..., ::31] *= 2.0 ** 10
    g = torch.Generator().manual_seed(n)
    q[:, :, 1::2] = q[:, :, 1::2] * 2.0 ** torch.randint(-6, 5, (B, n, hq // 2, D), generator=g).to(DEV)
    q = q.to(dtype)
    lens = [n + 20, 300]
    r = sd.attend(q, c.k, c.v, c.table, base._i32(lens), scale=scale, with_lse=True, **c.kw)
    torch.cuda.synchronize()
    assert not r["status"].any()
    for b, L in enumerate(lens):
        k, v = c.rows(b, L)
        out, lse, pv, av, qk = co.attend(base._np(q[b]), k, v, co.visible(n, n, L, 0, 0), scale)
        most = np.repeat(np.abs(k).sum(-1).max(0), hq // hkv)
        eq = scale * 2.0 ** -17 * np.abs(base._np(q[b])).max(-1) * most
        es = D * 2.0 ** -24 * qk + eq
        assert eq.max() < 1 / 32
        tol = ((2.0625 * es + 2.0 ** -13)[..., None] + base.U[F16]) * pv + 2.0 ** -25 * av + base.U[dtype] * np.abs(out) + 1e-30
        assert (np.abs(base._np(r["out"][b]) - out) <= tol).all(), (np.abs(base._np(r["out"][b]) - out).max(), tol.min())
        assert (np.abs(base._np(r["lse"][b]) - lse) <= es + 2.0 ** -13 + 2.0 ** -22 * np.abs(lse)).all()


@pytest.mark.parametrize("n", [3, 8, 40])
def test_queries_that_are_not_finite(sd, kernel, n):
    """An infinity or a NaN in a row of queries: the row is undefined, the others are not."""
    for dtype in (BF16, F16):
        c = Cache(1, 200, 32, 16, 2, 64)
        q = base._q(1, n, 8, 64, dtype)
        want = sd.attend(q, c.k, c.v, c.table, base._i32([200]), scale=0.01, with_lse=True, **c.kw)
        q[0, 1, 2, 5], q[0, 0, 7, 63], q[0, n - 1, 4, 0] = float("inf"), float("-inf"), float("nan")
        r = sd.attend(q, c.k, c.v, c.table, base._i32([200]), scale=0.01, with_lse=True, **c.kw)
        torch.cuda.synchronize()
        odd = torch.zeros(n, 8, dtype=torch.bool, device=DEV)
        odd[1, 2] = odd[0, 7] = odd[n - 1, 4] = True
        assert torch.isnan(r["out"][0][odd]).all() and torch.isnan(r["lse"][0][odd]).all()
        assert torch.equal(r["out"][0][~odd], want["out"][0][~odd]) and torch.equal(r["lse"][0][~odd], want["lse"][0][~odd])


def test_long_rows_split_over_the_gpu(sd, kernel):
    """Few rows over a long cache: many CTAs share a row, and their parts are joined."""
    c = Cache(1, 40000, 64, 64, 1, 128)
    base._run(sd, c, base._q(1, 1, 2, 128, F16), [39999], F16, 128, scale=0.05)
    c = Cache(3, 9000, 64, 16, 2, 64)
    base._run(sd, c, base._q(3, 3, 4, 64, BF16), [9000, 3, 5001], BF16, 64, scale=0.05)
    c = Cache(2, 3000, 64, 16, 1, 128)
    base._run(sd, c, base._q(2, 12, 2, 128, BF16), [3000, 1111], BF16, 128, scale=0.05)


@pytest.mark.parametrize("hkv,G,n,D", [(19, 2, 3, 64), (20, 1, 5, 64), (161, 1, 2, 64), (40, 1, 2, 128)])
def test_key_heads_that_do_or_do_not_divide_the_gpu(sd, kernel, hkv, G, n, D):
    lens = [700, 0, 33, 260, 129]
    c = Cache(len(lens), max(lens), 16, 16, hkv, D)
    base._run(sd, c, base._q(len(lens), n, hkv * G, D, BF16), lens, BF16, D, nq=[min(n, L) for L in lens], scale=0.05)


def test_many_short_sequences(sd, kernel):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 700).tolist()
    nq = [min(L, int(rng.integers(0, 3))) for L in lens]
    c = Cache(700, 40, 16, 16, 1, 64)
    base._run(sd, c, base._q(700, 2, 2, 64, BF16), lens, BF16, 64, nq=nq, scale=0.05)


def test_prompt_chunks(sd, kernel):
    c = Cache(2, 700, 32, 16, 1, 64)
    base._run(sd, c, base._q(2, 300, 3, 64, BF16), [700, 300], BF16, 64, what="chunk", scale=0.05)
    base._run(sd, c, base._q(2, 300, 3, 64, BF16), [700, 301], BF16, 64, window=130, sinks=5, what="window", scale=0.05)


def test_offsets_past_32_bits(sd, kernel):
    """A pool of more than 2^32 bytes, the sequence's pages at its end."""
    N, page, hkv, D = 140000, 64, 4, 128
    k = torch.zeros(N, page, hkv, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    v = torch.zeros(N, page, hkv, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ks, vs = (torch.zeros(N, 1, hkv, dtype=torch.uint8, device=DEV) for _ in range(2))
    c = Cache(1, 130, page, 64, hkv, D)
    far = torch.tensor([[N - 1, N - 5, N - 3]], dtype=torch.int32)
    for i in range(c.host_table.shape[1]):
        for dst, src in ((k, c.k), (v, c.v), (ks, c.ks), (vs, c.vs)):
            dst.view(torch.uint8)[int(far[0, i])] = src.view(torch.uint8)[int(c.host_table[0, i])]
    c.k, c.v, c.ks, c.vs, c.host_table, c.table = k, v, ks, vs, far, far.to(DEV)
    c.kw.update(k_scales=ks, v_scales=vs)
    c.N = N
    base._run(sd, c, base._q(1, 2, 8, D, BF16), [130], BF16, D, scale=0.05)
    new = _new(1, 20, hkv, D, BF16, std=20.0)
    before = c.codes("k", 0, 110)
    sd.append_kv8(new, new, c.k, c.v, c.table, base._i32([130]), **c.kw)
    r = sd.read_kv8(c.k, c.v, c.table, base._i32([130]), 20, **c.kw)
    torch.cuda.synchronize()
    assert (np.abs(base._np(r["k"]) - base._np(new)) <= (2.0 ** -4 + 2.0 ** -8) * np.abs(base._np(new)) + 0.02).all()
    assert np.array_equal(c.codes("k", 0, 64), before[:64])


def test_bad_pages_reach_the_rows_that_see_them(sd, kernel):
    """A page out of range gives NaN to the rows that see its slots, and to no others."""
    D, n = 64, 20
    c = Cache(2, 200, 16, 16, 2, D)
    c.table[0, 11] = c.N  # slots 176 .. 191 of sequence 0: its queries are slots 172 .. 191
    c.table[1, 0] = -7    # behind sequence 1's window
    q = base._q(2, n, 4, D, BF16)
    r = sd.attend(q, c.k, c.v, c.table, base._i32([192, 200]), window=60, scale=0.05, with_lse=True, **c.kw)
    torch.cuda.synchronize()
    assert r["status"].tolist() == [32, 0]
    assert torch.isfinite(r["out"][0, :4]).all() and torch.isnan(r["out"][0, 4:]).all() and torch.isnan(r["lse"][0, 4:]).all()
    assert torch.isfinite(r["out"][1]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 8, 40])
def test_a_pool_of_one_page_and_heads_at_one_place(sd, kernel, D, n):
    """Dimensions whose stride does not count, and one whose stride is zero: shared keys and values, or scales."""
    c = Cache(1, 100, 112, 16, 4, D, seed=n)
    p = int(c.host_table[0, 0])
    c.k, c.v, c.ks, c.vs = (t[p:p + 1] for t in (c.k, c.v, c.ks, c.vs))
    c.N, c.host_table, c.table = 1, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    c.kw.update(k_scales=c.ks, v_scales=c.vs)
    base._run(sd, c, base._q(1, n, 8, D, BF16), [100], BF16, D, what="one page", scale=0.05)
    c.k, c.v, c.ks, c.vs = (t[:, :, 1:2].expand(t.shape) for t in (c.k, c.v, c.ks, c.vs))
    c.kw.update(k_scales=c.ks, v_scales=c.vs)
    base._run(sd, c, base._q(1, n, 8, D, BF16), [100], BF16, D, what="one head", scale=0.05)


# ---- streams, graphs, repetition ------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 6, 40])
def test_same_bits_on_streams_and_from_graphs(sd, n):
    """Calls on a stream of their own, captured and replayed with other inputs in the same buffers, and two graphs
    replayed at once: the bits of an eager call."""
    B, hq, hkv, D = 4, 8, 2, 128
    c = Cache(B, 1200, 32, 32, hkv, D)
    lens = base._i32([n, 400, 1000, 1200])
    k, v, q = _new(B, n, hkv, D, BF16), _new(B, n, hkv, D, BF16, seed=9), base._q(B, n, hq, D, BF16)

    def step():
        a = sd.append_kv8(k, v, c.k, c.v, c.table, lens, **c.kw)
        r = sd.attend(q, c.k, c.v, c.table, lens, scale=0.05, with_lse=True, **c.kw)
        g = sd.read_kv8(c.k, c.v, c.table, lens, n, **c.kw)
        return {**r, "k": g["k"], "append": a["status"]}

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = sd.attend(q, c.k, c.v, c.table, lens, scale=0.05, with_lse=True, stream=side, **c.kw)
    side.synchronize()
    assert torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for s, g in zip((side, torch.cuda.Stream()), graphs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o["out"], want["out"]) and torch.equal(o["k"], want["k"])
    q2 = base._q(B, n, hq, D, BF16, seed=77)
    q.copy_(q2)
    lens.copy_(base._i32([n + 3, 399, 64 + n, 1100]))
    k.mul_(0.5)
    graphs[0].replay()
    torch.cuda.synchronize()
    again = step()
    torch.cuda.synchronize()
    assert torch.equal(outs[0]["out"], again["out"]) and torch.equal(outs[0]["k"], again["k"])
