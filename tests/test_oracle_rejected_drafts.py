"""What a rejected draft leaves in a block of an 8-bit cache, by the definition of the append (CPU): bounded as the header says,
and nothing where the block is put back before the accepted tokens are appended again."""
import numpy as np
import pytest

from oracle import cache_oracle as co


def _round(before, drafts, accepted, first, block, put_back):
    """Drafts [n, D] appended at slot `first`, of which the first `accepted` stay and are appended again."""
    codes, exps = co.append8(*before, drafts, first, block, 1.0)
    if put_back:
        lo = first // block
        codes[lo * block:(lo + 1) * block], exps[lo] = before[0][lo * block:(lo + 1) * block], before[1][lo]
    return co.append8(codes, exps, drafts[:accepted], first, block, 1.0)


@pytest.mark.parametrize("first", [3, 10, 16, 27])
@pytest.mark.parametrize("accepted", [0, 1, 4])
@pytest.mark.parametrize("raise_by", [1.0, 8.0, 300.0, 30000.0])
def test_marks_of_rejected_drafts(first, accepted, raise_by):
    block, D = 16, 64
    rng = np.random.default_rng(first + accepted)
    old = rng.normal(0, 1, (first, D)).astype(np.float32) * (2.0 ** rng.integers(-8, 3, (first, D))).astype(np.float32)
    drafts = rng.normal(0, 1, (8, D)).astype(np.float32)
    drafts[accepted:] *= raise_by
    follow = (rng.normal(0, 1, (3, D)) * 0.1).astype(np.float32)
    start = co.append8(np.full((64, D), 9, np.uint8), np.full(4, -3), old, 0, block, 1.0)
    end = first + accepted + len(follow)

    def finish(state):
        codes, exps = co.append8(*state, follow, first + accepted, block, 1.0)
        return codes[:end], np.repeat(exps, block)[:end, None]

    want = finish(co.append8(*start, drafts[:accepted], first, block, 1.0))  # a cache that never saw the rejected ones
    got = finish(_round(start, drafts, accepted, first, block, True))
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    got = finish(_round(start, drafts, accepted, first, block, False))
    a, b, scale = co.decode8(*got), co.decode8(*want), 2.0 ** got[1].astype(float)
    off = np.abs(a - b)
    assert (off <= 2.0 ** -9 * scale).all() and not off[np.abs(b) >= 2.0 ** -6 * scale].any()
    if raise_by > 100 and first % block:
        assert off.any()  # the mark is there
