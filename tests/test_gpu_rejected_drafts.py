"""Rejected drafts over 8-bit pages: what they leave in a block is bounded as include/specdec.h says, and a block that is put back
before the accepted tokens are appended again holds nothing of them."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import test_gpu_cache as base
import test_gpu_kv8 as kv8

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def sd(built_library):
    import speculative_decoding_token_temperature_gb300 as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def example(built_library):
    spec = importlib.util.spec_from_file_location("verify_round", ROOT / "examples" / "verify_round.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


NAMES = ("k", "v", "ks", "vs")


def _append(sd, c, k, v, lens, nq):
    r = sd.append_kv8(k, v, c.k, c.v, c.table, base._i32(lens), query_len=base._i32(nq), **c.kw)
    torch.cuda.synchronize()
    assert not r["status"].any()


def _state(c):
    return {w: getattr(c, w).view(torch.uint8).clone() for w in NAMES}


@pytest.mark.parametrize("page,block,hkv,D", [(64, 32, 2, 64), (48, 48, 1, 128), (32, 16, 3, 64)])
def test_a_cache_with_and_without_rejected_drafts(sd, page, block, hkv, D):
    """Accepted tokens, a round with rejected drafts 300 times as large, the next tokens: without them, with them, and with
    them and the first draft's block put back."""
    first, accepted, n = [5, 31, 32, 60, 77, 1], [0, 1, 3, 8, 2, 0], 8
    B = len(first)
    c = kv8.Cache(B, 120, page, block, hkv, D, seed=1)
    old_k, old_v = (kv8._new(B, 80, hkv, D, torch.float16, seed=s, spread=6, std=0.1) for s in (2, 3))
    _append(sd, c, old_k, old_v, first, first)
    start = _state(c)
    drafts = [kv8._new(B, n, hkv, D, torch.float16, seed=s) for s in (4, 5)]
    for b in range(B):
        for t in drafts:
            t[b, accepted[b]:] *= 300
    follow = [kv8._new(B, 3, hkv, D, torch.float16, seed=s, std=0.1) for s in (6, 7)]
    after = [f + a for f, a in zip(first, accepted)]
    got = {}
    for how in ("without", "with", "put back"):
        for w in NAMES:
            getattr(c, w).view(torch.uint8).copy_(start[w])
        if how != "without":
            _append(sd, c, *drafts, [f + n for f in first], [n] * B)
        if how == "put back":
            for b, f in enumerate(first):
                pg, blk = int(c.host_table[b, f // page]), f % page // block
                for w in "kv":
                    getattr(c, w).view(torch.uint8)[pg, blk * block:(blk + 1) * block] = start[w][pg, blk * block:(blk + 1) * block]
                    getattr(c, w + "s").view(torch.uint8)[pg, blk] = start[w + "s"][pg, blk]
        _append(sd, c, *drafts, after, accepted)
        _append(sd, c, *follow, [L + 3 for L in after], [3] * B)
        got[how] = [(c.codes(w, b, L + 3), c.exps(w, b, L + 3), x) for b, L in enumerate(after) for w, x in zip("kv", c.rows(b, L + 3))]
    marks = 0
    for (codes, exps, x), (codes1, exps1, x1), (codes2, exps2, x2) in zip(got["without"], got["with"], got["put back"]):
        assert np.array_equal(codes, codes2) and np.array_equal(exps, exps2)
        scale = 2.0 ** exps1[..., None] * 1.5  # (the larger of k_scale and v_scale)
        off = np.abs(x1 - x)
        assert (off <= 2.0 ** -9 * scale).all() and not off[np.abs(x) >= 2.0 ** -6 * scale].any()
        marks += int(off.any())
    assert marks > 0


def test_tree_rounds_do_not_depend_on_rejected_nodes(example):
    """Rounds whose random candidates differ and whose accepted tokens are the same leave the same cache, bit for bit."""
    B, prompt_len, left = 6, 37, []
    prompt = torch.randint(0, 1000, (B, prompt_len), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda", dtype=torch.int32)
    for seed in (0, 1, 2):
        model = example.ToyTarget(B=B, eight_bit=True, seed=3)
        emitted = example.rounds(model, prompt, [-1, -1, 0, 0, 2], 5, seed=seed)
        codes = []
        for b in range(B):
            slots = torch.arange(prompt_len + len(emitted[b]) - 1, device="cuda")  # (the last token's entry comes with the next round)
            page = model.table[b].long()[slots // 16]
            codes.append([(cache[w + "_pages"].view(torch.uint8)[page, slots % 16], cache[w + "_scales"][page]) for cache in model.cache for w in "kv"])
        left.append((emitted, codes))
    same = 0
    for emitted, codes in left[1:]:
        for b in range(B):
            if emitted[b] != left[0][0][b]:
                continue  # a random candidate was accepted
            same += 1
            for (x, s), (y, t) in zip(codes[b], left[0][1][b]):
                assert torch.equal(x, y) and torch.equal(s, t)
    assert same >= B


def test_compaction_moves_codes_and_appending_again_moves_values(sd):
    """compact_kv moves slots as bytes, as its documentation says: right for codes under one scale, not for blocks with scales of
    their own, whose accepted branch is appended again."""
    B, hkv, D, block, first, n = 1, 1, 64, 16, 16, 20
    c = kv8.Cache(B, 64, 32, block, hkv, D, seed=2)
    prefix = kv8._new(B, first, hkv, D, torch.float16, seed=3)
    _append(sd, c, prefix, prefix, [first], [first])
    nodes = kv8._new(B, n, hkv, D, torch.float16, seed=4)
    nodes[:, 16:] *= 64  # the nodes of the second block: another scale
    _append(sd, c, nodes, nodes, [first + n], [n])
    path = torch.tensor([[2, 7, 18]], dtype=torch.int32, device="cuda")
    before, start = c.codes("k", 0, first + n), _state(c)
    r = sd.compact_kv(c.k, base._i32([first]), path, base._i32([3]), block_table=c.table)
    torch.cuda.synchronize()
    assert r["new_len"].tolist() == [first + 3] and not r["status"].any()
    assert np.array_equal(c.codes("k", 0, first + 3), before[[*range(first), first + 2, first + 7, first + 18]])
    want = base._np(nodes[0, [2, 7, 18]])
    moved = c.rows(0, first + 3)[0][first:]
    assert np.abs(moved - want)[2].max() > 16 * np.abs(want[:2]).max()  # the large node's codes under a small node's scale
    for w in NAMES:
        getattr(c, w).view(torch.uint8).copy_(start[w])
    kept = nodes[:, [2, 7, 18]].contiguous()
    _append(sd, c, kept, kept, [first + 3], [3])
    for x in c.rows(0, first + 3):
        again = x[first:]
        assert (np.abs(again - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * np.abs(want).max()).all()
