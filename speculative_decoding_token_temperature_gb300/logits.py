"""What is done to the target's logits before they are verified: penalties for repeated tokens, biases
and grammar masks, for every row of a round, and the table of token counts they are computed from (the
logits calls of ``include/specdec.h``)."""
from __future__ import annotations

import ctypes

import torch

from . import cache as _cache

PROMPT = -2 ** 31  # a count's sign bit: the token is in the prompt


def declare(lib) -> None:
    """The argument types of the library's logits calls."""
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    lib.specdec_process_logits.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp]
    lib.specdec_count_tokens.argtypes = [vp, vp, i64, vp, i32, i32, i32, i32, i32, vp, vp]
    for f in (lib.specdec_process_logits, lib.specdec_count_tokens):
        f.restype = i32


def process_logits(logits, *, tokens=None, parents=None, gammas=None, counts=None, repetition=None, presence=None,
                   frequency=None, bias_tokens=None, bias_values=None, mask=None, out=None, stream=None) -> dict:
    """Penalties, biases and masks on the logits of a round (specdec_process_logits), whose result the
    verification calls take.

    logits [B, rows, V] bfloat16 or float32, the rows of a chain (row i follows drafts 0 .. i-1) or of a tree (row 0
    the root, row 1 + i node i); tokens [B, rows - 1] int32: the drafts, or the nodes' tokens, which count in
    the rows that follow them; parents [rows - 1] int32: a tree's (None: a chain); gammas [B] int32: the drafts that
    ``verify_chain_varlen`` verifies, rows past them are left alone; counts [B, V] int32: ``count_tokens``'s table of
    each sequence's tokens so far; repetition, presence, frequency [B] float32 (None: 1, 0 and 0); bias_tokens [B, n] int32
    (negative: skipped) and bias_values [B, n] float32; mask [B, rows, ceil(V / 32)] int32: bit t % 32 of word
    t // 32 is set where token t is allowed; out: a tensor like logits, or logits itself (in place).
    Returns logits [B, rows, V] and status [B]; the rows of a sequence in error are NaN."""
    call = (_cache._calls or _cache._module()).process_logits
    if stream is None:
        return call(logits, tokens, parents, gammas, counts, repetition, presence, frequency, bias_tokens, bias_values, mask, out)
    with torch.cuda.stream(stream):
        return call(logits, tokens, parents, gammas, counts, repetition, presence, frequency, bias_tokens, bias_values, mask, out)


def count_tokens(counts, tokens, *, num_tokens=None, prompt: bool = False, reset: bool = False, stream=None) -> dict:
    """Tokens added to the table of counts that ``process_logits`` reads (specdec_count_tokens), in place.

    counts [B, V] int32: how often each sequence generated a token, and in the sign bit whether its prompt has it;
    tokens [B, n] int32, a view with contiguous rows, of which num_tokens[b] (int32; None: all) count and negative ones are
    skipped: a verification call's ``tokens`` can be passed as they are; prompt: they are the prompt's; reset: the
    sequences' entries are set to zero before.  Returns counts and status [B]."""
    call = (_cache._calls or _cache._module()).count_tokens
    if stream is None:
        return call(counts, tokens, num_tokens, prompt, reset)
    with torch.cuda.stream(stream):
        return call(counts, tokens, num_tokens, prompt, reset)
