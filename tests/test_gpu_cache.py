"""GPU parity of the cache calls (rotation with the page write, 4-bit pages, attention over
pages) against the fp64 oracle, at the sizes, masks, strides and contents where they can go
wrong.

Tolerances, each derived from where a value is rounded.  u = eps/2 of the 16-bit type (bf16
2^-8, fp16 2^-11), and of fp16 for the weights of 4-bit pages.
  attention: a score is an fp32 sum of D products, off by at most D 2^-24 sum |q_d k_d|; its
    exponential (2^-22 with the scaling) and the running sums (2^-24 a term, at most 2^-13 for
    the lengths here) add to every weight's relative error, twice (the weight and the sum);
    the weight is rounded once more (u_w, and 2^-25 absolute where fp16 weights are
    subnormal), the output once (u).  4-bit pages with bf16 queries: q is held to 2^-25 of its
    row's largest value, below D 2^-24 of the products' sum for the vectors here.
  rotation: fp32 norm, angle (2^-25 turns and 2^-22 of sine and cosine) and products: 2^-20
    of |y_a| + |y_b|, then u of the value.
  4-bit codes and scales: exact.  Values read back: one rounding, u.
"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from oracle import specdec_oracle as so

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


@pytest.fixture(autouse=True, params=["rule", "warp", "tensor_memory"])
def kernel(request, hooks):
    """Every case through the kernel that the rule picks, and through each kernel."""
    hooks(attend_kernel=("rule", "warp", "tensor_memory").index(request.param))
    return request.param


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Cache:
    """Pages of B sequences in a shuffled order, their contents random."""

    def __init__(self, B, max_len, page, hkv, D, dtype, four=False, seed=0, layout="slots", std=1.0):
        g = torch.Generator().manual_seed(seed)
        per = max(1, -(-max_len // page))
        self.N, self.page, self.dtype, self.four = B * per + 3, page, dtype, four
        self.host_table = torch.randperm(self.N, generator=g)[:B * per].view(B, per).to(torch.int32)
        self.table = self.host_table.to(DEV)
        shape = (self.N, page, hkv, D)
        if four:
            mk = lambda d, lo, hi: torch.randint(lo, hi, (*shape[:3], d), generator=g, dtype=torch.uint8).to(DEV)  # noqa: E731
            self.k, self.v = mk(D // 2, 0, 256), mk(D // 2, 0, 256)
            self.ks, self.vs = mk(D // 16, 0x20, 0x40), mk(D // 16, 0x20, 0x40)
            self.kw = dict(k_scales=self.ks, v_scales=self.vs, k_scale=0.375, v_scale=1.5)
        else:
            self.kw = {}
            if layout == "slots":  # [pages, page, heads, D]
                self.k = (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)
                self.v = torch.randn(shape, generator=g).to(dtype).to(DEV)
            elif layout == "fused":  # keys and values of a page in one tensor
                both = (torch.randn(self.N, 2, page, hkv, D, generator=g) * std).to(dtype).to(DEV)
                self.k, self.v = both[:, 0], both[:, 1]
            else:  # heads outermost in a page, rows padded
                mk2 = lambda: (torch.randn(self.N, hkv, page, D + 8, generator=g) * std).to(dtype).to(DEV)[..., :D].permute(0, 2, 1, 3)  # noqa: E731
                self.k, self.v = mk2(), mk2()

    def rows(self, b, L):
        """Sequence b's first L slots as float64 [L, Hkv, D] keys and values."""
        s = torch.arange(L)
        at = (self.host_table[b].long()[s // self.page].to(DEV), (s % self.page).to(DEV))
        if self.four:
            return (co.dequantise(self.k[at].cpu().numpy(), self.ks[at].cpu().numpy(), self.kw["k_scale"]),
                    co.dequantise(self.v[at].cpu().numpy(), self.vs[at].cpu().numpy(), self.kw["v_scale"]))
        return _np(self.k[at]), _np(self.v[at])

    def put(self, which, b, slot, value):
        getattr(self, which)[int(self.host_table[b, slot // self.page]), slot % self.page] = value


def _check(got, got_lse, want, dtype, four, D, what=""):
    out, lse, pv, av, qk = want
    uw = U[torch.float16] if four else U[dtype]
    es = D * 2.0 ** -24 * qk
    rel = (2 * es + 2.0 ** -13)[..., None] + uw
    small = 2.0 ** -25 if (four or dtype == torch.float16) else 0.0
    tol = rel * pv + small * av + U[dtype] * np.abs(out) + 1e-30
    got = _np(got)
    nan = np.isnan(out)
    assert np.array_equal(np.isnan(got), nan), (what, np.argwhere(np.isnan(got) != nan)[:4])
    fin = np.isfinite(out)
    assert np.array_equal(got[~fin & ~nan], out[~fin & ~nan]), what
    bad = np.abs(got - out)[fin] > tol[fin]
    assert not bad.any(), (what, np.abs(got - out)[fin].max(), tol[fin].min(), bad.mean())
    if got_lse is not None:
        g = _np(got_lse)
        assert np.array_equal(np.isneginf(g), np.isneginf(lse)), what
        f = np.isfinite(lse)
        assert (np.abs(g - lse)[f] <= (es + 2.0 ** -13 + 2.0 ** -22 * np.abs(lse))[f]).all(), what
        assert np.array_equal(np.isnan(g), np.isnan(lse)), what


def _tree(n, seed):
    rng = np.random.default_rng(seed)
    parents = [-1] + [int(rng.integers(-1, i)) for i in range(1, n)]
    mask, depth, _ = so.build_tree_mask(parents, 0)
    return np.asarray(mask).astype(np.uint8), np.asarray(depth).astype(np.int32), parents


def _run(sd, c, q, lens, dtype, D, *, nq=None, window=0, sinks=0, mask=None, depth=None, scale=None, what="", **kw):
    n = q.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    r = sd.attend(q, c.k, c.v, c.table, _i32(lens), query_len=None if nq is None else _i32(nq), window=window, sinks=sinks,
                  tree_mask=None if mask is None else torch.tensor(mask, device=DEV),
                  depth=None if depth is None else torch.tensor(depth, device=DEV), scale=scale, with_lse=True, **c.kw, **kw)
    torch.cuda.synchronize()
    assert not r["status"].any(), (what, r["status"])
    for b, L in enumerate(lens):
        qn = n if nq is None else nq[b]
        k, v = c.rows(b, L)
        sees = co.visible(n, qn, L, window, sinks, mask, depth)
        _check(r["out"][b], r["lse"][b], co.attend(_np(q[b]), k, v, sees, scale), dtype, c.four, D, f"{what} b={b}")
    return r


def _q(B, n, hq, D, dtype, seed=1, std=1.0):
    return (torch.randn(B, n, hq, D, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).to(DEV)


# ---- attention ----------------------------------------------------------------------------

@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,D,n", [(8, 8, 64, 1), (8, 2, 128, 1), (16, 2, 128, 2), (7, 1, 64, 3), (12, 3, 128, 8),
                                        (28, 4, 128, 5), (4, 1, 64, 33), (10, 2, 128, 13), (40, 2, 64, 7)])
def test_chain_over_ragged_lengths(sd, four, dtype, hq, hkv, D, n):
    lens = [n, n + 1, 15 + n, 16 + n, 17 + n, 127 + n, 128 + n, 129 + n, 400 + n]
    c = Cache(len(lens), max(lens), 16, hkv, D, dtype, four, seed=n)
    _run(sd, c, _q(len(lens), n, hq, D, dtype, std=2.0), lens, dtype, D)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,n", [(1, 8), (1, 9), (1, 16), (1, 32), (1, 33), (3, 43), (1, 129), (2, 128), (1, 257), (5, 77)])
def test_row_tiles(sd, four, D, hq, n):
    """Query rows of a key head at and around the row tiles' borders (8, 32, 128, 256 rows), over one
    tile of 128 slots, two and several."""
    lens = [n, n + 100, n + 128, n + 500]
    c = Cache(len(lens), max(lens), 16, 1, D, torch.float16, four, seed=n)
    _run(sd, c, _q(len(lens), n, hq, D, torch.float16), lens, torch.float16, D)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("page", [1, 7, 24, 64, 500])
def test_pages_that_end_inside_a_step(sd, four, page):
    lens = [1, 6, 8, 63, 65, 333]
    c = Cache(len(lens), max(lens), page, 2, 128, torch.bfloat16, four, seed=page)
    _run(sd, c, _q(len(lens), 1, 8, 128, torch.bfloat16), lens, torch.bfloat16, 128)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (5, 1), (16, 16), (17, 4), (100, 40), (100000, 7), (64, 200)])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_window_and_sinks(sd, four, window, sinks, n):
    lens = [n, n + 3, n + 30, n + 155, n + 300]
    c = Cache(len(lens), max(lens), 16, 2, 64, torch.float16, four, seed=window)
    _run(sd, c, _q(len(lens), n, 6, 64, torch.float16), lens, torch.float16, 64, window=window, sinks=sinks)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("n,window,sinks", [(5, 0, 0), (17, 0, 0), (64, 0, 0), (64, 6, 2), (30, 3, 0), (2, 1, 1)])
def test_tree_masks(sd, four, n, window, sinks):
    lens = [n, n + 1, n + 29, n + 200]
    mask, depth, parents = _tree(n, n)
    built = sd.build_tree_mask(_i32(parents), 0)  # the framework's own mask and depth give the same
    c = Cache(len(lens), max(lens), 32, 2, 128, torch.bfloat16, four, seed=n)
    q = _q(len(lens), n, 8, 128, torch.bfloat16)
    r = _run(sd, c, q, lens, torch.bfloat16, 128, mask=mask, depth=depth, window=window, sinks=sinks)
    s = sd.attend(q, c.k, c.v, c.table, _i32(lens), tree_mask=built["mask"], depth=built["depth"], window=window, sinks=sinks,
                  **c.kw)
    assert torch.equal(r["out"], s["out"])


def test_rows_that_see_nothing_and_tokens_that_do_not_exist(sd):
    n, D = 6, 64
    mask = np.tril(np.ones((n, n), np.uint8))
    mask[0] = mask[4] = 0  # with no prefix these rows are empty
    lens, nq = [6, 4, 0, 9, 40], [6, 4, 0, 6, 0]
    for four in (False, True):
        c = Cache(5, 40, 8, 2, D, torch.bfloat16, four)
        r = _run(sd, c, _q(5, n, 4, D, torch.bfloat16), lens, torch.bfloat16, D, nq=nq, mask=mask)
        assert not r["out"][0, 0].any() and torch.isneginf(r["lse"][0, 4]).all()
        assert not r["out"][2].any() and not r["out"][4].any() and not r["out"][1, 4:].any()


@pytest.mark.parametrize("layout", ["fused", "heads"])
def test_strided_pages_and_queries(sd, layout):
    lens, D = [5, 100, 260], 128
    c = Cache(3, 260, 16, 4, D, torch.bfloat16, layout=layout)
    wide = _q(3, 5, 8 + 8, D, torch.bfloat16)
    _run(sd, c, wide[:, :, 8:], lens, torch.bfloat16, D)  # queries inside a fused projection's output
    turned = _q(3, 8, 5, D, torch.bfloat16).transpose(1, 2)  # heads before tokens
    _run(sd, c, turned, lens, torch.bfloat16, D)


def test_four_bit_pages_strided(sd):
    c = Cache(3, 260, 16, 4, 64, torch.float16, True)
    wide = [torch.zeros(c.N, 16, 6, w, dtype=torch.uint8, device=DEV) for w in (32, 32, 4, 4)]
    views = [w[:, :, 1:5] for w in wide]
    for dst, src in zip(views, (c.k, c.v, c.ks, c.vs)):
        dst.copy_(src)
    c.k, c.v, c.ks, c.vs = views
    c.kw.update(k_scales=c.ks.view(torch.float8_e4m3fn), v_scales=c.vs.view(torch.float8_e4m3fn))
    _run(sd, c, _q(3, 3, 8, 64, torch.float16), [3, 77, 260], torch.float16, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 8, 24])
def test_masked_slots_may_hold_anything(sd, dtype, n):
    """NaN and infinities behind the window, past the length, and in nodes that a row does not
    see stay out of its result; rows that do see them get what the formula gives."""
    D, window, sinks = 128, 40, 2
    lens = [n + 100, n + 7]
    c = Cache(2, max(lens) + 20, 16, 2, D, dtype)
    for b, L in enumerate(lens):
        for s in list(range(sinks, L - n - window)) + list(range(L, L + 20)):
            for which, val in (("k", float("nan")), ("v", float("inf") if s % 2 else float("nan"))):
                c.put(which, b, s, val)
    _run(sd, c, _q(2, n, 8, D, dtype), lens, dtype, D, window=window, sinks=sinks, what="outside")
    # a later draft's key and value are NaN: only the rows that see it are touched
    c.put("v", 0, lens[0] - 1, float("inf"))
    if n > 2:
        c.put("v", 0, lens[0] - 2, float("nan"))
        c.put("k", 1, lens[1] - 2, float("nan"))
    r = _run(sd, c, _q(2, n, 8, D, dtype), lens, dtype, D, window=window, sinks=sinks, what="inside")
    if n > 2:
        assert torch.isfinite(r["out"][0, :n - 2]).all() and torch.isnan(r["out"][0, n - 1]).all()


@pytest.mark.parametrize("n", [1, 8])
def test_masked_four_bit_groups_may_be_nan(sd, n):
    D, L = 128, 60 + n
    c = Cache(1, L + 20, 16, 2, D, torch.bfloat16, True)
    for s in range(L, L + 20):
        c.put("ks", 0, s, 0x7f)
        c.put("vs", 0, s, 0xff)
    c.vs[int(c.host_table[0, (L - 1) // 16]), (L - 1) % 16, :, 3] = 0x7f  # 16 values of the last draft
    r = _run(sd, c, _q(1, n, 8, D, torch.bfloat16), [L], torch.bfloat16, D)
    assert torch.isnan(r["out"][0, n - 1, :, 48:64]).all() and torch.isfinite(r["out"][0, n - 1, :, :48]).all()
    assert torch.isfinite(r["out"][0, :n - 1]).all()


def test_large_scores_and_scales(sd):
    for dtype, std in ((torch.bfloat16, 1e4), (torch.float16, 60.0)):
        lens = [3, 90]
        c = Cache(2, 90, 16, 1, 64, dtype, std=std)
        _run(sd, c, _q(2, 2, 4, 64, dtype, std=std), lens, dtype, 64, scale=0.0, what="scale 0")
        _run(sd, c, _q(2, 2, 4, 64, dtype, std=1e-3), lens, dtype, 64, scale=-0.5, what="negative scale")
    # 4-bit pages: bf16 queries far beyond fp16's range, and far below it
    c = Cache(2, 90, 16, 1, 64, torch.bfloat16, True)
    for std in (1e30, 1e-30, 0.0):
        _run(sd, c, _q(2, 2, 4, 64, torch.bfloat16, std=std), [3, 90], torch.bfloat16, 64, scale=0.0 if std == 0 else 0.01 / std,
             what=f"queries of {std}")


def test_long_rows_split_over_the_gpu(sd):
    """Few rows over a long cache: many CTAs share a row, and their parts are joined."""
    for four in (False, True):
        c = Cache(1, 40000, 64, 1, 128, torch.float16, four)
        _run(sd, c, _q(1, 1, 2, 128, torch.float16), [39999], torch.float16, 128)
        c = Cache(3, 9000, 64, 2, 64, torch.bfloat16, four)
        _run(sd, c, _q(3, 3, 4, 64, torch.bfloat16), [9000, 3, 5001], torch.bfloat16, 64)


def test_many_short_sequences(sd):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 700).tolist()
    nq = [min(L, int(rng.integers(0, 3))) for L in lens]
    c = Cache(700, 40, 8, 1, 64, torch.bfloat16)
    _run(sd, c, _q(700, 2, 2, 64, torch.bfloat16), lens, torch.bfloat16, 64, nq=nq)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("hkv,G,n,D", [(19, 2, 3, 64), (20, 1, 5, 64), (161, 1, 2, 64), (40, 1, 2, 128)])
def test_key_heads_that_do_or_do_not_divide_the_gpu(sd, four, hkv, G, n, D):
    lens = [700, 0, 33, 260, 129]
    dtype = torch.bfloat16
    c = Cache(len(lens), max(lens), 16, hkv, D, dtype, four)
    _run(sd, c, _q(len(lens), n, hkv * G, D, dtype), lens, dtype, D, nq=[min(n, L) for L in lens])


def test_prompt_chunks(sd):
    for four in (False, True):
        c = Cache(2, 700, 32, 1, 64, torch.bfloat16, four)
        _run(sd, c, _q(2, 300, 3, 64, torch.bfloat16), [700, 300], torch.bfloat16, 64, what="chunk")
        _run(sd, c, _q(2, 300, 3, 64, torch.bfloat16), [700, 301], torch.bfloat16, 64, window=130, sinks=5, what="window")


def test_offsets_past_32_bits(sd):
    """A pool of more than 2^32 bytes, the sequence's pages at its end."""
    N, page, hkv, D = 70000, 64, 4, 128
    k = torch.zeros(N, page, hkv, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    c = Cache(1, 130, page, hkv, D, torch.bfloat16)
    far = torch.tensor([[N - 1, N - 5, N - 3]], dtype=torch.int32)
    for i in range(c.host_table.shape[1]):
        k[int(far[0, i])] = c.k[int(c.host_table[0, i])]
        v[int(far[0, i])] = c.v[int(c.host_table[0, i])]
    c.k, c.v, c.host_table, c.table = k, v, far, far.to(DEV)
    _run(sd, c, _q(1, 2, 8, D, torch.bfloat16), [130], torch.bfloat16, D)


def test_bad_lengths_and_pages(sd):
    """Data errors are found by the host or by the kernels' own range checks: reported for the
    sequence, nothing outside the pages is read."""
    D, n = 64, 3
    for four in (False, True):
        c = Cache(7, 96, 16, 2, D, torch.bfloat16, four)
        t = c.table.clone()
        t[1, 1], t[2, 0], t[3, 5] = c.N, -1, 1 << 30
        lens = [50, 50, 50, 60, 97, 2, -1]  # 3: its bad page lies past its length; 4: past the table; 5: fewer than n
        q = _q(7, n, 4, D, torch.bfloat16)
        r = sd.attend(q, c.k, c.v, t, _i32(lens), with_lse=True, **c.kw)
        torch.cuda.synchronize()
        assert r["status"].tolist() == [0, 32, 32, 0, 32, 32, 32]
        assert torch.isnan(r["out"][[1, 2, 4, 5, 6]]).all() and torch.isnan(r["lse"][[1, 2, 4, 5, 6]]).all()
        assert torch.isfinite(r["out"][[0, 3]]).all()
        # behind a window nobody looks at the entry
        r = sd.attend(q, c.k, c.v, t, _i32(lens), window=8, **c.kw)
        torch.cuda.synchronize()
        assert r["status"].tolist() == [0, 0, 0, 0, 32, 32, 32] and torch.isfinite(r["out"][:4]).all()
        # the first slots are seen: sequence 2's page 0 counts again
        r = sd.attend(q, c.k, c.v, t, _i32(lens), window=8, sinks=1, **c.kw)
        torch.cuda.synchronize()
        assert r["status"].tolist() == [0, 0, 32, 0, 32, 32, 32] and torch.isnan(r["out"][2]).all()


def test_same_inputs_give_the_same_bits_and_streams(sd):
    lens = [700, 1300, 9]
    c = Cache(3, 1300, 16, 2, 128, torch.bfloat16)
    q = _q(3, 8, 8, 128, torch.bfloat16)
    a = sd.attend(q, c.k, c.v, c.table, _i32(lens), with_lse=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    L = _i32(lens)
    torch.cuda.synchronize()
    for _ in range(3):
        b = sd.attend(q, c.k, c.v, c.table, L, with_lse=True, stream=side)
        side.synchronize()
        assert all(torch.equal(a[x], b[x]) for x in a)


def test_two_streams_at_a_time(sd):
    """Calls on two streams, whose launches and workspaces may overlap, give what one gives."""
    cases = []
    for seed, n, L in ((1, 8, 3000), (2, 40, 2000)):
        c = Cache(4, L, 16, 2, 128, torch.bfloat16, seed=seed)
        cases.append((c, _q(4, n, 8, 128, torch.bfloat16, seed=seed), _i32([L, L // 2, n, L - 7])))
    want = [sd.attend(q, c.k, c.v, c.table, lens, with_lse=True) for c, q, lens in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for i, (c, q, lens) in enumerate(cases):
            got[i].append(sd.attend(q, c.k, c.v, c.table, lens, with_lse=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(r[x], want[i][x]) for x in r)


def test_captured_in_a_graph(sd):
    lens = _i32([100, 260])
    c = Cache(2, 320, 16, 2, 64, torch.float16)
    q, k, v = (_q(2, 4, h, 64, torch.float16, seed=h) for h in (6, 2, 2))
    turns = sd.rotation_turns([1.0 / 10 ** (j / 8) for j in range(16)], DEV)

    def step():
        r = sd.rotate_qk(q, k, turns, lens, v=v, k_pages=c.k, v_pages=c.v, block_table=c.table)
        return sd.attend(r["q"], c.k, c.v, c.table, lens)["out"]

    want = step().clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for extra in (0, 60):
        lens += extra
        g.replay()
        torch.cuda.synchronize()
        if not extra:
            assert torch.equal(out, want)
    eager = step()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)  # the replay followed the lengths


# ---- rotation -------------------------------------------------------------------------------

def _rotate_check(got, x, pos, freq, w, dtype, interleaved, eps=1e-6):
    want = co.rotate(x, pos, freq, w, eps, interleaved)
    mag = np.abs(want).copy()
    half = len(freq)
    a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    mag[a] = mag[b] = np.hypot(want[a], want[b]) * 2 ** 0.5
    tol = U[dtype] * np.abs(want) + (2.0 ** -20 + U[dtype] * 2.0 ** -11) * mag + (2.0 ** -25 if dtype == torch.float16 else 0)
    assert (np.abs(got - want) <= tol).all(), (pos, np.abs(got - want).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 32, True), (128, 128, False), (128, 128, True),
                                               (128, 48, False), (64, 16, False)])
@pytest.mark.parametrize("paged,norm", [(True, True), (False, True), (True, False)])
def test_rotation_matches_the_oracle(sd, dtype, D, rot, interleaved, paged, norm):
    B, n, hq, hkv = 4, 5, 6, 2
    lens, nq = [5, 333, 70, 4], [5, 5, 3, 0]
    fused = _q(B, n, hq + 2 * hkv, D, dtype, std=3.0)
    q, k, v = fused[:, :, :hq], fused[:, :, hq:hq + hkv], fused[:, :, hq + hkv:]
    freq = [10000.0 ** (-2 * j / rot) for j in range(rot // 2)]
    wq, wk = (_q(1, 1, 1, D, dtype, seed=s).view(D) if norm else None for s in (5, 6))
    c = Cache(B, 350, 16, hkv, D, dtype)
    before = c.k.clone(), c.v.clone()
    kw = dict(v=v, k_pages=c.k, v_pages=c.v, block_table=c.table) if paged else {}
    r = sd.rotate_qk(q, k, sd.rotation_turns(freq, DEV), _i32(lens), query_len=_i32(nq), q_weight=wq, k_weight=wk,
                     interleaved=interleaved, **kw)
    torch.cuda.synchronize()
    assert not r["status"].any()
    written = torch.zeros(c.N, 16, dtype=torch.bool)
    for b in range(B):
        for i in range(n):
            if i >= nq[b]:
                assert not r["q"][b, i].any()
                if not paged:
                    assert not r["k"][b, i].any()
                continue
            s = lens[b] - nq[b] + i
            for h in range(hq):
                _rotate_check(_np(r["q"][b, i, h]), _np(q[b, i, h]), s, freq, None if wq is None else _np(wq), dtype, interleaved)
            pg, off = int(c.host_table[b, s // 16]), s % 16
            written[pg, off] = True
            for h in range(hkv):
                got = c.k[pg, off, h] if paged else r["k"][b, i, h]
                _rotate_check(_np(got), _np(k[b, i, h]), s, freq, None if wk is None else _np(wk), dtype, interleaved)
            if paged:
                assert torch.equal(c.v[pg, off], v[b, i])
    keep = (~written).to(DEV)
    if paged:
        assert torch.equal(c.k[keep], before[0][keep]) and torch.equal(c.v[keep], before[1][keep])


def test_rotation_at_far_positions_and_tree_depths(sd):
    freq = [500000.0 ** (-2 * j / 64) for j in range(32)]
    D, n = 64, 4
    depth = [0, 1, 1, 2]
    lens = [4, 1 << 20, (1 << 31) - 1, 123456789]
    q, k = _q(4, n, 2, D, torch.float16), _q(4, n, 1, D, torch.float16, seed=4)
    r = sd.rotate_qk(q, k, sd.rotation_turns(freq, DEV), _i32(lens), depth=_i32(depth))
    torch.cuda.synchronize()
    for b, L in enumerate(lens):
        for i in range(n):
            for x, y in ((q, r["q"]), (k, r["k"])):
                # the frequency itself is a float64 (2^-53): at 2^31 positions that is 2^-22 of a radian
                _rotate_check(_np(y[b, i, 0]), _np(x[b, i, 0]), L - n + depth[i], freq, None, torch.float16, False)


def test_rotation_bad_sequences_are_left_alone(sd):
    B, n, D = 5, 3, 64
    q, k = _q(B, n, 4, D, torch.bfloat16), _q(B, n, 2, D, torch.bfloat16, seed=2)
    c = Cache(B, 64, 16, 2, D, torch.bfloat16)
    t = c.table.clone()
    t[1, 1], t[2, 0] = -7, c.N
    before = c.k.clone()
    lens = [20, 17, 20, 65, 2]  # 1: its last new token is on the bad page; 2: the bad page holds no new token
    r = sd.rotate_qk(q, k, sd.rotation_turns([1.0] * 32, DEV), _i32(lens), v=k, k_pages=c.k, v_pages=c.v, block_table=t)
    torch.cuda.synchronize()
    assert r["status"].tolist() == [0, 32, 0, 32, 32]
    assert torch.isnan(r["q"][[1, 3, 4]]).all() and torch.isfinite(r["q"][[0, 2]]).all()
    changed = (c.k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) == {int(c.host_table[0, 1]), int(c.host_table[2, 1])}


# ---- 4-bit pages ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,hkv,page", [(64, 1, 16), (128, 3, 7)])
def test_four_bit_codes_scales_and_values(sd, dtype, D, hkv, page):
    B, n = 3, 9
    lens, nq = [9, 30, 21], [9, 4, 0]
    k, v = _q(B, n, hkv, D, dtype, std=2.0), _q(B, n, hkv, D, dtype, seed=9)
    k[0, 0, 0, :16] = 0
    k[0, 1, 0, :16] = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, .75, .25, -6, -5, -3.5, -2.5, -1.75, -1.25, -.75, -.25]) * 0.5
    k[0, 2, 0, 3], k[0, 3, 0, 20], v[0, 4, 0, 50] = float("nan"), float("inf"), float("-inf")
    k[0, 5, 0, :16] = 60000.0
    v[0, 6, 0, :16] = 2.0 ** -14
    c = Cache(B, 30, page, hkv, D, dtype, True)
    c.kw.update(k_scale=0.5, v_scale=0.37)
    before = [x.clone() for x in (c.k, c.v, c.ks, c.vs)]
    st = sd.append_kv4(k, v, c.k, c.v, c.table, _i32(lens), query_len=_i32(nq), **c.kw)["status"]
    r = sd.read_kv4(c.k, c.v, c.table, _i32(lens), n, query_len=_i32(nq), dtype=dtype, **c.kw)
    torch.cuda.synchronize()
    assert not st.any() and not r["status"].any()
    written = torch.zeros(c.N, page, dtype=torch.bool)
    for b in range(B):
        for i in range(nq[b]):
            s = lens[b] - nq[b] + i
            pg, off = int(c.host_table[b, s // page]), s % page
            written[pg, off] = True
            for x, codes, scales, ts, back in ((k, c.k, c.ks, 0.5, r["k"]), (v, c.v, c.vs, 0.37, r["v"])):
                for h in range(hkv):
                    row = x[b, i, h].float().cpu().numpy()
                    want = [co.quantise_group(row[g:g + 16], ts) for g in range(0, D, 16)]
                    assert scales[pg, off, h].tolist() == [w[1] for w in want], (b, i, h)
                    nib = np.concatenate([w[0] for w in want])
                    packed = nib[0::2] | (nib[1::2] << 4)
                    assert codes[pg, off, h].tolist() == packed.tolist(), (b, i, h)
                    val = co.dequantise(packed, scales[pg, off, h].cpu().numpy(), ts)
                    got = _np(back[b, i, h])
                    assert np.array_equal(np.isnan(got), np.isnan(val))
                    ok = np.isfinite(val) & (np.abs(val) < torch.finfo(dtype).max)
                    small = 2.0 ** -25 if dtype == torch.float16 else 0.0
                    # the two fp32 products before the rounding: 2^-23 each
                    assert (np.abs(got - val)[ok] <= (U[dtype] + 2.0 ** -22) * np.abs(val)[ok] + small).all()
        assert not r["k"][b, nq[b]:].any() and not r["v"][b, nq[b]:].any()
    keep = (~written).to(DEV)
    for x, y in zip((c.k, c.v, c.ks, c.vs), before):
        assert torch.equal(x[keep], y[keep])


def test_four_bit_signs_of_zero_and_quotients_next_to_ties(sd):
    """The codes are those of the IEEE quotient: -0 keeps its sign, and values a step of the type on
    either side of a tie go to either side of it."""
    n, hkv, D, dtype = 64, 2, 64, torch.float16
    k, v = _q(1, n, hkv, D, dtype, std=3.0), torch.zeros(1, n, hkv, D, device=DEV, dtype=dtype)
    k[0, :, :, 1::5], v[0, :, :, ::2] = -0.0, -0.0
    ties = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    steps = torch.nextafter(ties.to(dtype), torch.tensor(float("inf"), dtype=dtype)), torch.nextafter(ties.to(dtype), torch.tensor(0.0, dtype=dtype))
    for i in range(n):
        m = 6 * (1 + (i % 8) / 8) * 2.0 ** (i // 8 - 6)  # each mantissa of the scale
        v[0, i, 0, :16] = torch.cat([torch.tensor([m, -m], dtype=torch.float64), *(x.double() * m / 6 for x in steps)]).to(dtype).to(DEV)
    c = Cache(1, n, 16, hkv, D, dtype, True)
    sd.append_kv4(k, v, c.k, c.v, c.table, _i32([n]), **c.kw)
    torch.cuda.synchronize()
    for x, codes, scales, ts in ((k, c.k, c.ks, c.kw["k_scale"]), (v, c.v, c.vs, c.kw["v_scale"])):
        for i in range(n):
            pg, off = int(c.host_table[0, i // 16]), i % 16
            for h in range(hkv):
                row = x[0, i, h].float().cpu().numpy()
                want = [co.quantise_group(row[g:g + 16], ts) for g in range(0, D, 16)]
                nib = np.concatenate([w[0] for w in want])
                assert scales[pg, off, h].tolist() == [w[1] for w in want], (i, h)
                assert codes[pg, off, h].tolist() == (nib[0::2] | (nib[1::2] << 4)).tolist(), (i, h)


def test_four_bit_bad_sequences(sd):
    c = Cache(3, 40, 16, 2, 64, torch.bfloat16, True)
    t = c.table.clone()
    t[1, 2] = c.N
    k = _q(3, 3, 2, 64, torch.bfloat16)
    before = [x.clone() for x in (c.k, c.v, c.ks, c.vs)]
    lens = _i32([41 + 8, 35, 2])
    st = sd.append_kv4(k, k, c.k, c.v, t, lens, **c.kw)["status"]
    r = sd.read_kv4(c.k, c.v, t, lens, 3, **c.kw)
    torch.cuda.synchronize()
    assert st.tolist() == [32, 32, 32] and r["status"].tolist() == [32, 32, 32]
    assert torch.isnan(r["k"]).all() and torch.isnan(r["v"]).all()
    assert all(torch.equal(x, y) for x, y in zip((c.k, c.v, c.ks, c.vs), before))


def test_attention_reads_what_append_wrote(sd):
    """Write, attend, compact: the same pages through the framework's calls."""
    B, n, hq, hkv, D, page = 2, 5, 4, 2, 64, 16
    lens = [37, 16]
    c = Cache(B, 48, page, hkv, D, torch.bfloat16, True)
    k, v, q = (_q(B, n, h, D, torch.bfloat16, seed=s) for h, s in ((hkv, 1), (hkv, 2), (hq, 3)))
    sd.append_kv4(k, v, c.k, c.v, c.table, _i32(lens), **c.kw)
    back = sd.read_kv4(c.k, c.v, c.table, _i32(lens), n, dtype=torch.float16, **c.kw)
    _run(sd, c, q, lens, torch.bfloat16, D)
    # the branch of nodes 1 and 3 moves to the first new slots, in codes and scales alike
    path, acc = _i32([[1, 3]] * B), _i32([2] * B)
    prefix = _i32([L - n for L in lens])
    for t in (c.k, c.v, c.ks, c.vs):
        sd.compact_kv(t, prefix, path, acc, block_table=c.table)
    kept = sd.read_kv4(c.k, c.v, c.table, prefix + 2, 2, dtype=torch.float16, **c.kw)
    torch.cuda.synchronize()
    assert torch.equal(kept["k"], back["k"][:, [1, 3]]) and torch.equal(kept["v"], back["v"][:, [1, 3]])
