"""fp64 CPU oracle of the logits calls -- test infrastructure only: one row and one token's count at a time, from
the definitions in ``include/specdec.h``."""
from __future__ import annotations

import numpy as np


def paths(n: int, parents=None) -> list:
    """For each row of n drafts (n + 1 rows), the drafts it follows: a chain, or a tree's root paths."""
    out = [[]]
    for i in range(n):
        out.append(out[1 + (i - 1 if parents is None else int(parents[i]))] + [i])
    return out


def process(logits, tokens=None, parents=None, counts=None, repetition=1.0, presence=0.0, frequency=0.0, bias=(), mask=None):
    """One sequence: logits [rows, V] float64, tokens [rows - 1], counts [V] (the sign bit: prompt), bias a list of
    (token, value), mask [rows, words].  Returns the processed rows and, for tolerances, the sum of the magnitudes
    that its roundings are relative to."""
    x = np.asarray(logits, np.float64)
    rows, V = x.shape
    out, size = np.empty_like(x), np.empty_like(x)
    base = np.zeros(V, np.int64) if counts is None else np.asarray(counts, np.int64)
    prompt, base = base < 0, base & 0x7FFFFFFF
    b = np.zeros(V)
    for t, v in bias:
        if t >= 0:
            b[t] = v
    follows = paths(rows - 1, parents) if tokens is not None else [[]] * rows
    for i in range(rows):
        c = base.copy()
        for j in follows[i]:
            c[tokens[j]] += 1
        with np.errstate(invalid="ignore", over="ignore"):
            y = np.where(prompt | (c > 0), np.where(x[i] > 0, x[i] / repetition, x[i] * repetition), x[i])
            pen = frequency * c + np.where(c > 0, presence, 0.0)
            out[i] = y - pen + b
            size[i] = np.abs(y) + np.abs(pen) + np.abs(b - pen) + np.abs(out[i])
        if mask is not None:
            bits = (np.asarray(mask[i]).astype(np.int64)[:, None] >> np.arange(32)) & 1
            out[i][bits.reshape(-1)[:V] == 0] = -np.inf
    return out, size


def count(counts, tokens, prompt: bool = False, reset: bool = False):
    """One sequence's table [V] after its tokens (negative ones, and those past the vocabulary, skipped)."""
    out = np.zeros_like(counts) if reset else np.array(counts)
    for t in tokens:
        if 0 <= t < len(out):
            out[t] = out[t] | np.int32(-2 ** 31) if prompt else out[t] + 1
    return out
