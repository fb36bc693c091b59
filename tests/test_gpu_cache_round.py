"""Rounds of tree verification around the paged cache (examples/verify_round.py): speculation over
the pages emits what decoding token by token over the same pages emits."""
import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def example(built_library):
    spec = importlib.util.spec_from_file_location("verify_round", ROOT / "examples" / "verify_round.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _greedy(model, prompt, count):
    B = prompt.shape[0]
    length = torch.full((B,), prompt.shape[1], dtype=torch.int32, device=prompt.device)
    out = [model.step(prompt, length)[:, -1].argmax(-1).to(torch.int32)]
    for _ in range(count):
        length = length + 1
        out.append(model.step(out[-1][:, None], length)[:, 0].argmax(-1).to(torch.int32))
    return torch.stack(out, 1).tolist()


@pytest.mark.parametrize("four_bit,window,sinks", [(False, 0, 0), (True, 0, 0), (False, 24, 4)])
def test_tree_rounds_emit_what_greedy_decoding_emits(example, four_bit, window, sinks):
    """Greedy decoding and tree rounds see the same prefixes; their scores differ in rounding only, so a
    token may differ where two logits are near: the common prefix covers at least the first
    rounds for most requests, and the whole for some."""
    kw = dict(B=6, four_bit=four_bit, window=window, sinks=sinks, seed=3)
    prompt = torch.randint(0, 1000, (6, 37), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda", dtype=torch.int32)
    spec = example.rounds(example.ToyTarget(**kw), prompt, [-1, -1, 0, 0, 2], 5)
    plain = _greedy(example.ToyTarget(**kw), prompt, 12)
    same = []
    for s, p in zip(spec, plain):
        assert len(s) >= 6 + 5  # every round accepts the target's own choice, and emits one more
        n = min(len(s), len(p))
        same.append(next((i for i in range(n) if s[i] != p[i]), n) / n)
    assert sum(x == 1.0 for x in same) >= 3 and sorted(same)[1] >= 0.25, same
