"""Rounds over 8-bit pages with processed logits: the calls one after another, as a server makes them, each held to its
oracle on what the calls before it left; and the example of whole tree rounds."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import test_gpu_cache as base
import test_gpu_kv8 as kv8
import test_gpu_logits as logits
from oracle import cache_oracle as co
from oracle import logits_oracle as lo
from oracle import specdec_oracle as so

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
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


def test_chain_rounds(sd):
    """Drafts written to the pages, attended to, their logits penalised, biased and masked, verified for a number of drafts of each
    request's own, counted; the next round goes on from the accepted lengths."""
    B, gamma, hq, hkv, D, V = 5, 4, 4, 2, 64, 512
    rows = gamma + 1
    rng = np.random.default_rng(7)
    c = kv8.Cache(B, 200, 32, 32, hkv, D, seed=5)
    unembed = base._q(1, hq * D, 1, V, torch.bfloat16, seed=2, std=0.08)[0, :, 0]
    prompt = torch.randint(0, V, (B, 40), generator=torch.Generator().manual_seed(1), dtype=torch.int32).to(DEV)
    counts = torch.full((B, V), 77, dtype=torch.int32, device=DEV)
    sd.count_tokens(counts, prompt, prompt=True, reset=True)
    table = np.stack([lo.count(np.zeros(V, np.int32), prompt[b].tolist(), prompt=True) for b in range(B)])
    rep, pres, freq = (torch.tensor(rng.uniform(a, b, B), dtype=torch.float32, device=DEV) for a, b in ((1.0, 1.5), (0, 0.5), (0, 0.3)))
    bias_tokens = torch.tensor(rng.integers(0, V, (B, 6)), dtype=torch.int32, device=DEV)
    bias_values = torch.tensor(rng.normal(0, 2, (B, 6)), dtype=torch.float32, device=DEV)
    lens = [40] * B
    for step in range(4):
        drafts = torch.tensor(rng.integers(0, V, (B, gamma)), dtype=torch.int32, device=DEV)
        drafts[:, 1] = prompt[:, step]
        lens = [L + rows for L in lens]
        kv8._append_and_check(sd, c, kv8._new(B, rows, hkv, D, torch.bfloat16, seed=step, std=2.0 ** step),
                              kv8._new(B, rows, hkv, D, torch.bfloat16, seed=99 + step), lens)
        q = base._q(B, rows, hq, D, torch.bfloat16, seed=step)
        r = base._run(sd, c, q, lens, torch.bfloat16, D, what=f"round {step}")
        x = {"logits": (r["out"].reshape(B, rows, hq * D) @ unembed).contiguous(), "tokens": drafts, "counts": counts, "repetition": rep,
             "presence": pres, "frequency": freq, "bias_tokens": bias_tokens, "bias_values": bias_values,
             "mask": torch.tensor(rng.integers(-2 ** 31, 2 ** 31, (B, rows, V // 32)), dtype=torch.int32, device=DEV)}
        gammas = base._i32(rng.integers(0, gamma + 1, B).tolist())
        p = sd.process_logits(x["logits"], gammas=gammas, **{k: v for k, v in x.items() if k != "logits"})
        torch.cuda.synchronize()
        assert not p["status"].any()
        for b in range(B):
            n = int(gammas[b]) + 1
            one = {k: v[b:b + 1, :n] if k in ("logits", "mask") else v[b:b + 1, :n - 1] if k == "tokens" else v[b:b + 1] for k, v in x.items()}
            logits._check(p["logits"][b:b + 1, :n], one, f"round {step} b={b}")
        qd = torch.softmax(torch.tensor(rng.normal(0, 2, (B, gamma, V)), dtype=torch.float32, device=DEV), -1)
        temps, u = torch.ones(B, device=DEV), torch.tensor(rng.random((B, rows)), dtype=torch.float32, device=DEV)
        v = sd.verify_chain_varlen(p["logits"], qd, drafts, temps, u, gammas)
        torch.cuda.synchronize()
        for b in range(B):
            n = int(gammas[b])
            f = p["logits"][b].float().cpu().numpy()
            f[n + 1:] = 0
            want = so.verify_chain_varlen_sequence(f, qd[b].cpu().numpy(), drafts[b].cpu().numpy(), 1.0, u[b].cpu().numpy(), n)
            assert v["tokens"][b].tolist() == want["tokens"].tolist(), (step, b)
        sd.count_tokens(counts, v["tokens"])
        torch.cuda.synchronize()
        accepted = v["num_accepted"].tolist()
        for b in range(B):
            table[b] = lo.count(table[b], v["tokens"][b].tolist())
            lens[b] += accepted[b] + 1 - rows  # (the extra token's entry comes with the next round)
        assert np.array_equal(counts.cpu().numpy(), table)


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 4)])
def test_tree_rounds_over_eight_bit_pages(example, window, sinks):
    """Whole rounds run: every round accepts the target's own choice and emits one more."""
    model = example.ToyTarget(B=6, eight_bit=True, window=window, sinks=sinks, seed=3)
    prompt = torch.randint(0, 1000, (6, 37), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda", dtype=torch.int32)
    emitted = example.rounds(model, prompt, [-1, -1, 0, 0, 2], 5)
    assert all(len(e) >= 6 + 5 and all(0 <= t < 1000 for t in e) for e in emitted)


def test_penalised_tree_rounds_do_not_repeat(example):
    """Under a penalty that leaves no repeated token near the others, a request's tokens differ from each other and from its prompt's."""
    for eight in (False, True):
        model = example.ToyTarget(B=4, eight_bit=eight, seed=4)
        prompt = torch.randint(0, 1000, (4, 30), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda", dtype=torch.int32)
        emitted = example.rounds(model, prompt, [-1, -1, 0, 0, 2], 6, repetition=1e6)
        for b, e in enumerate(emitted):
            assert len(set(e)) == len(e) >= 12 and not set(e) & set(prompt[b].tolist()), (eight, b)
