"""GPU parity of the logits calls (penalties, biases, masks; the table of counts) against the fp64 oracle.

Tolerance of a processed logit: the quotient or product, the penalty (one fused rounding), its difference from the bias
and the last sum are each rounded once in fp32: 2^-24 of their own magnitudes, whose sum the oracle gives; a bf16 result is rounded
once more, 2^-8 of itself.  Counts are exact.
"""
import numpy as np
import pytest
import torch

from oracle import logits_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _parents(n, seed):
    rng = np.random.default_rng(seed)
    return [int(rng.integers(-1, i)) for i in range(n)]


def _case(B, rows, V, dtype, seed=0, counts=True, penalties=True, bias=0, mask=False, tokens=True, tree=False):
    """Inputs of the call: drafts that repeat and that are in the history, biases listed twice and skipped."""
    g = torch.Generator().manual_seed(seed)
    x = {"logits": (torch.randn(B, rows, V, generator=g) * 4).to(dtype)}
    small = max(1, min(V, 40))
    if tokens and rows > 1:
        t = torch.randint(0, small, (B, rows - 1), generator=g, dtype=torch.int32)
        t[:, ::3] = torch.randint(0, V, (B, rows - 1), generator=g, dtype=torch.int32)[:, ::3]
        t[:, -1] = V - 1
        x["tokens"] = t
        if tree:
            x["parents"] = torch.tensor(_parents(rows - 1, seed), dtype=torch.int32)
    if counts:
        c = (torch.rand(B, V, generator=g) < 0.3).int() * torch.randint(1, 9, (B, V), generator=g, dtype=torch.int32)
        x["counts"] = torch.where(torch.rand(B, V, generator=g) < 0.2, c - 2 ** 31, c).int()
    if penalties:
        x["repetition"] = 0.5 + torch.rand(B, generator=g) * 1.5
        x["presence"] = torch.randn(B, generator=g)
        x["frequency"] = torch.randn(B, generator=g)
    if bias:
        bt = torch.randint(-1, V, (B, bias), generator=g, dtype=torch.int32)
        bt[:, bias // 2:] = torch.where(torch.rand(B, bias - bias // 2, generator=g) < 0.3, bt[:, :1], bt[:, bias // 2:])
        x["bias_tokens"], x["bias_values"] = bt, torch.randn(B, bias, generator=g) * 5
    if mask:
        m = torch.randint(-2 ** 31, 2 ** 31, (B, rows, (V + 31) // 32), generator=g)
        m[:, rows // 2] = 0      # a row whose mask leaves nothing
        m[:, 0] = -1             # and one that allows everything
        x["mask"] = m.to(torch.int32)
    return {k: v.to(DEV) for k, v in x.items()}


def _expect(x, b):
    rows = x["logits"].shape[1]
    get = lambda k: None if k not in x else x[k][b].cpu().numpy()  # noqa: E731
    num = lambda k, d: d if k not in x else float(x[k][b])  # noqa: E731
    bias = [] if "bias_tokens" not in x else list(zip(x["bias_tokens"][b].tolist(), x["bias_values"][b].double().tolist()))
    return lo.process(_np(x["logits"][b]), tokens=get("tokens"), parents=None if "parents" not in x else x["parents"].tolist(), counts=get("counts"),
                      repetition=num("repetition", 1.0), presence=num("presence", 0.0), frequency=num("frequency", 0.0), bias=bias,
                      mask=None if "mask" not in x else x["mask"][b].cpu().numpy())[:2] + (rows,)


def _check(got, x, what=""):
    dtype = x["logits"].dtype
    for b in range(got.shape[0]):
        want, size, _ = _expect(x, b)
        y = _np(got[b])
        assert np.array_equal(np.isnan(y), np.isnan(want)), what
        odd = ~np.isfinite(want)
        assert np.array_equal(y[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)]), what
        tol = 2.0 ** -24 * 1.01 * size + (2.0 ** -8 * np.abs(want) if dtype == BF16 else 0) + 1e-40
        bad = np.abs(y - want)[~odd] > tol[~odd]
        assert not bad.any(), (what, b, np.argwhere((np.abs(y - want) > tol) & ~odd)[:4], np.abs(y - want)[~odd].max())


def _run(sd, x, **kw):
    r = sd.process_logits(x["logits"], **{k: v for k, v in x.items() if k != "logits"}, **kw)
    torch.cuda.synchronize()
    assert not r["status"].any()
    return r["logits"]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 7, 8, 31, 33, 1000, 2048, 2049, 4104, 5003])
@pytest.mark.parametrize("rows", [1, 2, 9])
def test_everything_at_odd_and_even_sizes(sd, dtype, V, rows):
    x = _case(3, rows, V, dtype, seed=V + rows, bias=6, mask=True)
    _check(_run(sd, x), x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 6001, 9000])
@pytest.mark.parametrize("drop", ["counts", "penalties", "bias", "mask", "tokens", "all"])
def test_each_part_may_be_missing(sd, dtype, V, drop):
    kw = dict(counts=True, penalties=True, bias=4, mask=True, tokens=True)
    for k in kw:
        if drop in (k, "all"):
            kw[k] = False if k != "bias" else 0
    x = _case(2, 5, V, dtype, seed=V, **kw)
    got = _run(sd, x)
    _check(got, x, drop)
    if drop == "all":
        assert torch.equal(got, x["logits"])


@pytest.mark.parametrize("missing", [("repetition",), ("presence", "frequency"), ("repetition", "presence")])
def test_each_penalty_may_be_missing(sd, missing):
    x = _case(2, 4, 2500, BF16, bias=3)
    for k in missing:
        del x[k]
    _check(_run(sd, x), x, str(missing))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,V", [(2, 100), (65, 3001), (65, 4096), (300, 513)])
def test_trees(sd, dtype, rows, V):
    x = _case(2, rows, V, dtype, seed=rows, bias=5, mask=True, tree=True)
    _check(_run(sd, x), x)


def test_many_rows_of_a_chain(sd):
    x = _case(1, 256, 700, BF16, bias=2)
    _check(_run(sd, x), x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [4000, 4001])
def test_in_place_and_into_a_buffer(sd, dtype, V):
    x = _case(3, 4, V, dtype, bias=4, mask=True)
    want = _run(sd, x)
    out = torch.empty_like(x["logits"])
    r = _run(sd, x, out=out)
    assert r.data_ptr() == out.data_ptr() and torch.equal(r, want)
    y = x["logits"].clone()
    kw = {k: v for k, v in x.items() if k != "logits"}
    r = sd.process_logits(y, out=y, **kw)["logits"]
    torch.cuda.synchronize()
    assert r.data_ptr() == y.data_ptr() and torch.equal(y, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [512, 515])
def test_logits_that_are_not_finite(sd, dtype, V):
    """Infinities and NaN follow the formula, and a masked place is -inf whatever it holds."""
    x = _case(2, 3, V, dtype, bias=3, mask=True)
    x["logits"][:, :, ::5] = float("nan")
    x["logits"][:, :, 1::5] = float("inf")
    x["logits"][:, :, 2::5] = float("-inf")
    x["logits"][:, :, 3::5] = 0.0
    _check(_run(sd, x), x)
    x["bias_values"][:] = float("-inf")  # a ban
    x["logits"][:, :, 1::5] = 1.0
    _check(_run(sd, x), x)


def test_unaligned_views(sd):
    """Logits and results that start anywhere on their elements."""
    for dtype in (BF16, F32):
        x = _case(2, 3, 800, dtype, bias=3, mask=True)
        want = _run(sd, x)
        n = x["logits"].numel()
        for off_in, off_out in ((1, 0), (0, 1), (3, 2)):
            src = torch.empty(n + 8, dtype=dtype, device=DEV)[off_in:off_in + n].view(2, 3, 800)
            src.copy_(x["logits"])
            dst = torch.empty(n + 8, dtype=dtype, device=DEV)[off_out:off_out + n].view(2, 3, 800)
            assert torch.equal(_run(sd, {**x, "logits": src}, out=dst), want)


@pytest.mark.parametrize("V", [2000, 2001])
def test_rows_past_a_requests_drafts_are_left_alone(sd, V):
    B, rows = 4, 6
    x = _case(B, rows, V, BF16, bias=3, mask=True)
    want = _run(sd, x)
    gammas = [0, 5, 2, 3]
    x["tokens"][0, 0:] = -1   # tokens past the counts may hold anything
    x["tokens"][2, 2:] = V
    out = torch.full_like(x["logits"], 7.0)
    r = _run(sd, x, gammas=_i32(gammas), out=out)
    for b, gam in enumerate(gammas):
        assert torch.equal(r[b, :gam + 1], want[b, :gam + 1]) and (r[b, gam + 1:] == 7.0).all()


def test_errors_are_reported_for_their_sequence(sd):
    B, rows, V = 12, 4, 3000
    x = _case(B, rows, V, F32, bias=3, mask=True)
    want = _run(sd, x)
    x["tokens"][1, 2] = -1
    x["tokens"][2, 0] = V
    x["bias_tokens"][3, 1] = V
    x["repetition"][4] = 0.0
    x["repetition"][5] = float("inf")
    x["repetition"][6] = float("nan")
    x["presence"][7] = float("inf")
    x["frequency"][8] = float("nan")
    x["repetition"][9] = -1.0
    r = sd.process_logits(x["logits"], **{k: v for k, v in x.items() if k != "logits"})
    torch.cuda.synchronize()
    assert r["status"].tolist() == [0, 4, 4, 4, 64, 64, 64, 64, 64, 64, 0, 0]
    assert torch.isnan(r["logits"][1:10]).all()
    for b in (0, 10, 11):
        assert torch.equal(r["logits"][b], want[b])
    x = _case(3, rows, V, BF16)
    r = sd.process_logits(x["logits"], tokens=x["tokens"], gammas=_i32([-1, 4, 3]))
    torch.cuda.synchronize()
    assert r["status"].tolist() == [4, 4, 0] and torch.isnan(r["logits"][:2]).all()
    for bad in ([0, 0, 0], [-2, 0, 0], [-1, 0, 2]):
        r = sd.process_logits(x["logits"], tokens=x["tokens"], parents=_i32(bad))
        torch.cuda.synchronize()
        assert r["status"].tolist() == [32, 32, 32] and torch.isnan(r["logits"]).all(), bad


def test_wrong_arguments_raise(sd):
    x = _case(2, 3, 100, BF16, bias=3, mask=True)
    lg = x["logits"]
    for kw in (dict(tokens=x["tokens"][:, :1]), dict(tokens=x["tokens"].long()), dict(tokens=x["tokens"].cpu()), dict(parents=_i32([-1, 0])),
               dict(counts=x["counts"][:, :50]), dict(repetition=x["repetition"].double()), dict(bias_tokens=x["bias_tokens"]),
               dict(bias_tokens=x["bias_tokens"], bias_values=x["bias_values"][:, :2]), dict(mask=x["mask"][:, :, :3]), dict(mask=x["mask"].long()),
               dict(out=lg.float()), dict(out=lg[:1]), dict(tokens=x["tokens"], parents=_i32([-1, 0]), gammas=_i32([1, 1]))):
        with pytest.raises(ValueError):
            sd.process_logits(lg, **kw)
    c = torch.zeros(2, 50, dtype=torch.int32, device=DEV)
    for kw in (dict(counts=c, tokens=_i32([[1], [2], [3]])), dict(counts=c.long(), tokens=_i32([[1], [2]])), dict(counts=c.t(), tokens=_i32([[1], [2]])),
               dict(counts=c, tokens=_i32([[1], [2]]).long()), dict(counts=c, tokens=_i32([[1, 2], [2, 3]]).t()),
               dict(counts=c, tokens=_i32([[1], [2]]), num_tokens=_i32([1]))):
        with pytest.raises(ValueError):
            sd.count_tokens(**kw)
    with pytest.raises(RuntimeError, match="ambiguous"):
        sd.count_tokens(c, _i32([[1], [2]]), prompt=torch.ones(2, dtype=torch.bool))
    torch.cuda.synchronize()
    assert not c.any()


# ---- the table ------------------------------------------------------------------------------

@pytest.mark.parametrize("V", [1, 100, 8192, 8193, 20000])
@pytest.mark.parametrize("n", [0, 1, 5, 255, 257, 3000])
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("reset", [False, True])
def test_counts(sd, V, n, prompt, reset):
    rng = np.random.default_rng(V + n)
    B = 3
    tokens = rng.integers(-1, max(1, V // 3), (B, n)).astype(np.int32)
    tokens[:, : n // 2] = rng.integers(0, V, (B, n // 2))
    old = rng.integers(0, 5, (B, V)).astype(np.int32)
    old[rng.random((B, V)) < 0.2] |= np.int32(-2 ** 31)
    num = [n, n // 2, 0]
    t = torch.tensor(old, device=DEV)
    r = sd.count_tokens(t, torch.tensor(tokens, device=DEV), num_tokens=_i32(num), prompt=prompt, reset=reset)
    torch.cuda.synchronize()
    assert not r["status"].any() and r["counts"].data_ptr() == t.data_ptr()
    for b in range(B):
        assert np.array_equal(t[b].cpu().numpy(), lo.count(old[b], tokens[b, :num[b]], prompt, reset)), b


def test_tokens_past_the_vocabulary_and_lengths_out_of_range(sd):
    V = 50
    for reset in (False, True):
        t = torch.zeros(5, V, dtype=torch.int32, device=DEV)
        tok = _i32([[1, 50, 2], [1, 1, 1], [-5, 3, 2 ** 31 - 1], [7, 8, 9], [49, 0, 50]])
        r = sd.count_tokens(t, tok, num_tokens=_i32([3, 9, 2, -4, 2]), reset=reset)
        torch.cuda.synchronize()
        assert r["status"].tolist() == [4, 0, 0, 0, 0]
        want = np.zeros((5, V), np.int32)
        want[0, [1, 2]] = 1
        want[1, 1], want[2, 3] = 3, 1
        want[4, [0, 49]] = 1
        assert np.array_equal(t.cpu().numpy(), want)


def test_strided_tokens_and_a_view_of_the_table(sd):
    t = torch.zeros(4, 100, dtype=torch.int32, device=DEV)
    wide = torch.arange(40, dtype=torch.int32, device=DEV).view(2, 20)
    sd.count_tokens(t[1:3], wide[:, 3:9])
    torch.cuda.synchronize()
    want = np.zeros((4, 100), np.int32)
    want[1, 3:9], want[2, 23:29] = 1, 1
    assert np.array_equal(t.cpu().numpy(), want)


@pytest.mark.parametrize("V", [3000, 3001])
def test_streams_and_graphs(sd, V):
    x = _case(3, 5, V, BF16, bias=4, mask=True)
    want = _run(sd, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw = {k: v for k, v in x.items() if k != "logits"}
    r = sd.process_logits(x["logits"], stream=side, **kw)["logits"]
    side.synchronize()
    assert torch.equal(r, want)
    table = torch.zeros(3, V, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.count_tokens(table, x["tokens"])
        out = sd.process_logits(x["logits"], **{**kw, "counts": table})
    table.zero_()
    for i in range(3):
        x["tokens"].copy_((x["tokens"] + 17) % V)
        g.replay()
    torch.cuda.synchronize()
    assert not out["status"].any() and int(table.sum()) == 3 * 4 * 3
    _check(out["logits"], {**x, "counts": table})


def test_outputs_that_overlap_the_logits_raise(sd):
    buf = torch.zeros(2 * 3 * 100 + 8, device=DEV)
    with pytest.raises(RuntimeError):
        sd.process_logits(buf[:600].view(2, 3, 100), out=buf[8:].view(2, 3, 100))


def test_many_rows_past_32_bits(sd):
    """The most rows, over more than 2^31 logits: each equals the row of a call of its own, whose counts hold the drafts."""
    B, rows, V = 2, 8192, 140001
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(B, rows, V, generator=g, device=DEV, dtype=BF16)
    t = torch.randint(0, V, (B, rows - 1), generator=g, device=DEV, dtype=torch.int32)
    t[:, ::5], t[:, -1] = 7, V - 1
    kw = dict(repetition=torch.tensor([1.5, 0.75], device=DEV), presence=torch.tensor([0.5, -1.0], device=DEV),
              frequency=torch.tensor([0.25, 0.125], device=DEV))
    r = sd.process_logits(x, tokens=t, **kw)
    assert not r["status"].any()
    for i in (0, 1, 2, 4096, rows - 2, rows - 1):
        counts = torch.zeros(B, V, dtype=torch.int32, device=DEV)
        for b in range(B):
            counts[b] = torch.bincount(t[b, :i].long(), minlength=V)[:V].int()
        assert torch.equal(sd.process_logits(x[:, i:i + 1].contiguous(), counts=counts, **kw)["logits"], r["logits"][:, i:i + 1]), i


@pytest.mark.parametrize("reset", [False, True])
def test_counts_past_32_bits(sd, reset):
    B, V = 17000, 128256
    counts = torch.full((B, V), 3 if reset else 0, dtype=torch.int32, device=DEV)
    t = torch.tensor([5, V - 1, 5], dtype=torch.int32, device=DEV).expand(B, 3)
    assert not sd.count_tokens(counts, t, reset=reset)["status"].any()
    assert (counts[:, 5] == 2).all() and (counts[:, V - 1] == 1).all()
    assert int(counts.sum(dtype=torch.int64)) == 3 * B
