"""One round of tree verification around the paged cache, with the library's calls only between the
projections: the step a serving loop repeats for every layer, and the round that ends it.

A toy target of a few layers runs a batch of candidate trees: the fused projection's queries and
keys are normed, rotated to the nodes' positions and written to the cache pages
(`rotate_qk`, or `append_kv4` where pages are held in 4 bits), the nodes attend over pages and
ancestors (`attend` with `build_tree_mask`), the logits of the last layer are verified
(`verify_tree`), and the accepted branch's entries are gathered (`compact_kv`).

    python examples/verify_round.py [--four-bit] [--window 256 --sinks 4]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_token_temperature_gb300 as sd  # noqa: E402


class ToyTarget:
    """Random weights of a small target: B requests, each with pages of its own."""

    def __init__(self, B=4, layers=2, heads=8, kv_heads=2, head_dim=64, vocab=1000, page=16, max_len=512, four_bit=False,
                 window=0, sinks=0, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        width = heads * head_dim
        rand = lambda *s: torch.empty(*s, device=device).normal_(0, s[-2] ** -0.5, generator=g).bfloat16()  # noqa: E731
        self.heads, self.kv_heads, self.D, self.four = heads, kv_heads, head_dim, four_bit
        self.window, self.sinks = window, sinks
        self.embed, self.unembed = rand(1, vocab, width)[0] * vocab ** 0.5, rand(width, vocab)
        self.qkv = [rand(width, (heads + 2 * kv_heads) * head_dim) for _ in range(layers)]
        self.out = [rand(width, width) for _ in range(layers)]
        self.q_norm, self.k_norm = (torch.ones(head_dim, device=device, dtype=torch.bfloat16) for _ in range(2))
        self.turns = sd.rotation_turns([10000.0 ** (-2 * j / head_dim) for j in range(head_dim // 2)], device)
        per = math.ceil(max_len / page)
        self.table = torch.randperm(B * per, generator=g, device=device).to(torch.int32).view(B, per)
        pages = (B * per, page, kv_heads)
        if four_bit:
            self.cache = [{n: torch.zeros(*pages, head_dim // (2 if "pages" in n else 16), device=device, dtype=torch.uint8)
                           for n in ("k_pages", "v_pages", "k_scales", "v_scales")} for _ in range(layers)]
            self.scales = {"k_scale": 0.5, "v_scale": 0.25}
        else:
            self.cache = [{n: torch.zeros(*pages, head_dim, device=device, dtype=torch.bfloat16) for n in ("k_pages", "v_pages")}
                          for _ in range(layers)]
            self.scales = {}

    def step(self, tokens, context_len, tree=None):
        """Logits [B, n, V] of the new tokens [B, n], whose entries the pages then hold; tree: the
        mask and depth of `build_tree_mask(parents, 0)` for nodes, None for consecutive tokens."""
        B, n = tokens.shape
        depth = tree["depth"] if tree else None
        x = self.embed[tokens.long()]
        for qkv, out, cache in zip(self.qkv, self.out, self.cache):
            y = (x @ qkv).view(B, n, self.heads + 2 * self.kv_heads, self.D)
            q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], 2)
            norms = {"q_weight": self.q_norm, "k_weight": self.k_norm, "depth": depth}
            if self.four:
                r = sd.rotate_qk(q, k, self.turns, context_len, **norms)
                sd.append_kv4(r["k"], v, cache["k_pages"], cache["v_pages"], self.table, context_len,
                              k_scales=cache["k_scales"], v_scales=cache["v_scales"], **self.scales)
            else:
                r = sd.rotate_qk(q, k, self.turns, context_len, v=v, block_table=self.table, **norms, **cache)
            o = sd.attend(r["q"], block_table=self.table, context_len=context_len, tree_mask=tree["mask"] if tree else None,
                          depth=depth, window=self.window, sinks=self.sinks, **cache, **self.scales)
            x = x + o["out"].view(B, n, -1) @ out
        return (x @ self.unembed).contiguous()

    def keep(self, prefix_len, path, num_accepted):
        """The accepted branch's entries move to consecutive slots, in every page tensor."""
        for cache in self.cache:
            for t in cache.values():
                r = sd.compact_kv(t, prefix_len, path, num_accepted, block_table=self.table)
        return r["new_len"]


def rounds(model, prompt, parents, count, seed=0):
    """Greedy rounds: the prompt's pass, then `count` trees of random candidates around the target's own
    choice.  Returns the emitted tokens of every request."""
    dev, B = prompt.device, prompt.shape[0]
    g = torch.Generator(device=dev).manual_seed(seed)
    n = len(parents)
    par = torch.tensor(parents, dtype=torch.int32, device=dev)
    tree = sd.build_tree_mask(par, 0)
    depth_max = int(tree["depth"].max()) + 1
    length = torch.full((B,), prompt.shape[1], dtype=torch.int32, device=dev)
    last = model.step(prompt, length)[:, -1].argmax(-1).to(torch.int32)
    emitted = [[int(t)] for t in last]
    for _ in range(count):
        # the root of the tree is the last emitted token (its entry is not in the cache yet); candidates
        # are random around the target's own choice here, a drafter's in earnest
        logits = model.step(last[:, None], length + 1)
        length = length + 1
        vocab = logits.shape[-1]
        nodes = torch.randint(0, vocab, (B, n), generator=g, device=dev, dtype=torch.int32)
        nodes[:, 0] = logits[:, 0].argmax(-1).to(torch.int32)
        rows = torch.cat((logits, model.step(nodes, length + n, tree)), 1)
        u = torch.zeros(B, depth_max + 1, device=dev)
        r = sd.verify_tree(rows, nodes, par, torch.zeros(B, device=dev), u, depth_max)
        length = model.keep(length, r["path"], r["num_accepted"])
        acc = r["num_accepted"].tolist()
        toks = r["tokens"].tolist()
        for b in range(B):
            emitted[b] += toks[b][:acc[b] + 1]
        last = torch.tensor([e[-1] for e in emitted], dtype=torch.int32, device=dev)
    return emitted


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--four-bit", action="store_true")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    a = ap.parse_args()
    model = ToyTarget(four_bit=a.four_bit, window=a.window, sinks=a.sinks)
    prompt = torch.randint(0, 1000, (4, 37), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.int32)
    for b, e in enumerate(rounds(model, prompt, [-1, -1, 0, 0, 2], 6)):
        print(f"request {b}: {len(e)} tokens in 6 rounds: {e}")


if __name__ == "__main__":
    main()
