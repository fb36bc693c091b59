"""More of the logits' processing against the fp64 oracle: in place and into other buffers without masks, where only the tokens that
change are touched; rows and neighbours that must stay as they are."""
import pytest
import torch

import test_gpu_logits as base

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


def _rest(x):
    return {k: v for k, v in x.items() if k != "logits"}


def _bits(t):
    return t.view(torch.int32 if t.dtype == F32 else torch.int16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 5, 2048, 4000, 4001])
@pytest.mark.parametrize("rows,tree", [(1, False), (4, False), (7, False), (7, True), (66, True)])
@pytest.mark.parametrize("bias", [0, 4])
def test_in_place_without_masks(sd, dtype, V, rows, tree, bias):
    """What a call into another tensor gives, and what the oracle does."""
    x = base._case(3, rows, V, dtype, seed=V + rows, bias=bias, tree=tree)
    want = base._run(sd, x)
    base._check(want, x)
    y = x["logits"].clone()
    r = sd.process_logits(y, out=y, **_rest(x))
    torch.cuda.synchronize()
    assert not r["status"].any() and r["logits"].data_ptr() == y.data_ptr()
    assert torch.equal(_bits(y), _bits(want))
    out = torch.full_like(x["logits"], 7.0)
    assert torch.equal(_bits(base._run(sd, x, out=out)), _bits(want))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [800, 801])
def test_unaligned_views_without_masks(sd, dtype, V):
    """Logits and results that start anywhere on their elements, alike on 16 bytes or not, and in place; what lies around them stays."""
    x = base._case(2, 3, V, dtype, bias=3)
    want, n = base._run(sd, x), x["logits"].numel()
    for off_in, off_out in ((1, 0), (0, 1), (3, 2), (1, 1), (5, 5)):
        src = torch.empty(n + 16, dtype=dtype, device=DEV)[off_in:off_in + n].view(2, 3, V)
        src.copy_(x["logits"])
        around = torch.full((n + 16,), 9.0, dtype=dtype, device=DEV)
        assert torch.equal(base._run(sd, {**x, "logits": src}, out=around[off_out:off_out + n].view(2, 3, V)), want)
        assert (around[:off_out] == 9.0).all() and (around[off_out + n:] == 9.0).all()
        around = torch.full((n + 16,), 9.0, dtype=dtype, device=DEV)
        place = around[off_in:off_in + n].view(2, 3, V)
        place.copy_(x["logits"])
        sd.process_logits(place, out=place, **_rest(x))
        torch.cuda.synchronize()
        assert torch.equal(place, want) and (around[:off_in] == 9.0).all() and (around[off_in + n:] == 9.0).all()


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("V", [2000, 2001])
def test_in_place_rows_past_a_requests_drafts_are_left_alone(sd, V, mask):
    B, rows = 4, 6
    x = base._case(B, rows, V, BF16, bias=3, mask=mask)
    want, gammas = base._run(sd, x), [0, 5, 2, 3]
    x["tokens"][0, 0:] = -1   # tokens past the counts may hold anything
    x["tokens"][2, 2:] = V
    y = x["logits"].clone()
    r = sd.process_logits(y, out=y, gammas=base._i32(gammas), **_rest(x))
    torch.cuda.synchronize()
    assert not r["status"].any()
    for b, gam in enumerate(gammas):
        assert torch.equal(y[b, :gam + 1], want[b, :gam + 1]) and torch.equal(_bits(y[b, gam + 1:]), _bits(x["logits"][b, gam + 1:]))


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [3000, 3001])
def test_in_place_errors_are_their_sequences_own(sd, dtype, V, mask):
    """The rows of a sequence in error are NaN, its neighbours' are what they would be."""
    B, rows = 7, 5
    x = base._case(B, rows, V, dtype, bias=3, mask=mask)
    want = base._run(sd, x)
    x["tokens"][1, 2] = -1
    x["bias_tokens"][3, 1] = V
    x["repetition"][5] = 0.0
    y = x["logits"].clone()
    r = sd.process_logits(y, out=y, **_rest(x))
    torch.cuda.synchronize()
    assert r["status"].tolist() == [0, 4, 0, 4, 0, 64, 0]
    for b in range(B):
        assert torch.isnan(y[b]).all() if b % 2 else torch.equal(_bits(y[b]), _bits(want[b])), b


def test_in_place_without_anything_to_change(sd):
    x = torch.randn(2, 3, 1001, device=DEV)
    y = x.clone()
    r = sd.process_logits(y, out=y)
    torch.cuda.synchronize()
    assert not r["status"].any() and torch.equal(x, y)
