"""Cases of the 8-bit cache and of the logits' processing: what is measured, on which inputs, and
what the outputs have to be.

The operators are the write of keys and values into cache pages held in 8 bits with a scale for
each block of tokens and head (`append_kv8`, read back by `read_kv8`), attention over such pages
(`attend`), and what is done to a verification round's logits before they are verified: penalties
for repeated tokens, biases and grammar masks, where every row has the drafts before it in its history
(`process_logits`), with the table of token counts that they read (`count_tokens`).  `run` computes them
in plain torch operations where `own` is false, and calls the framework where it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
LEAST, MOST = -15, 7   # exponents of a block's scale
PROMPT = -2 ** 31      # a count's sign bit: the token is in the prompt


# ---- the cases --------------------------------------------------------------------------

def _append8(name, B, n, hkv, d, dtype, ctx, page, block):
    return {"name": name, "op": "append8", "B": B, "n": n, "hkv": hkv, "d": d, "dtype": dtype, "ctx": ctx, "page": page,
            "block": block}


def _attend8(name, B, n, hq, hkv, d, dtype, ctx, page, block, window, sinks, tree):
    return {"name": name, "op": "attend8", "B": B, "n": n, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "ctx": ctx,
            "page": page, "block": block, "window": window, "sinks": sinks, "tree": tree}


def _process(name, B, rows, V, dtype, history, bias, mask, tree):
    return {"name": name, "op": "process", "B": B, "rows": rows, "V": V, "dtype": dtype, "history": history, "bias": bias,
            "mask": mask, "tree": tree}


def _count(name, B, n, V, prompt, reset):
    return {"name": name, "op": "count", "B": B, "n": n, "V": V, "prompt": prompt, "reset": reset}


def listed():
    return [
        # the 8-bit write of a verification round: 7 drafts and the bonus row, into blocks that hold tokens already
        _append8("append 8-bit verify", 64, 8, 8, 128, "bf16", 512, 64, 64),
        # the 8-bit write of prompts' chunks, an odd number of tokens, a scale for 16 tokens
        _append8("append 8-bit prompt", 4, 2045, 8, 128, "fp16", 2500, 32, 16),
        # one request, one token, a short cache: latency
        _attend8("attend 8-bit one token", 1, 1, 32, 8, 128, "bf16", 901, 64, 64, 0, 0, False),
        # one token of many requests over long ragged caches
        _attend8("attend 8-bit decode", 96, 1, 64, 8, 128, "fp16", 16001, 32, 16, 0, 0, False),
        # verification of 7 drafts and the bonus row
        _attend8("attend 8-bit verify", 64, 8, 32, 8, 128, "bf16", 8190, 64, 64, 0, 0, False),
        # the 64-node candidate tree of the tree verification workload
        _attend8("attend 8-bit tree", 24, 64, 32, 8, 128, "bf16", 12000, 64, 32, 0, 0, True),
        # a prompt's chunk with a window and first tokens that stay visible, heads of 64
        _attend8("attend 8-bit prompt", 2, 1100, 16, 2, 64, "fp16", 6001, 128, 128, 2048, 16, False),
        # one request's next token: latency
        _process("process one row", 1, 1, 32000, "fp32", 600, 0, False, False),
        # the benchmarked verification batch: 7 drafts and the bonus row, penalties and biases
        _process("process verify", 256, 8, 128256, "bf16", 4000, 300, False, False),
        # the tree workload under a grammar: a mask for every node, an odd vocabulary
        _process("process tree", 32, 65, 32001, "bf16", 1500, 16, True, True),
        # the history of a batch of prompts, from nothing
        _count("count prompts", 64, 4095, 128256, True, True),
        # one more chunk of a long prompt
        _count("count chunk", 4, 2048, 152064, True, False),
    ]


HEADS = ((32, 8, 128), (28, 4, 128), (40, 8, 64), (16, 2, 64), (64, 8, 128), (6, 6, 128), (8, 1, 128), (12, 12, 64))
VOCABS = (1000, 32000, 32001, 50257, 65024, 128256, 152064)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    op = rng.choice(("append8", "attend8", "attend8", "process", "process", "count"))
    most = {"append8": 1, "attend8": 5, "process": 8, "count": 10}
    limit = _cost(listed()[most[op]])
    while True:
        if op in ("append8", "attend8"):
            hq, hkv, d = rng.choice(HEADS)
            dtype = rng.choice(("bf16", "fp16"))
            page = rng.choice((16, 32, 48, 64, 128, 256))
            block = rng.choice([b for b in (16, 32, 48, 64, 128, 256) if page % b == 0])
            B = _log_int(rng, 1, 128)
        if op == "append8":
            n = _log_int(rng, 1, 2800)
            case = _append8("", B, n, hkv, d, dtype, n + rng.randint(0, 700), page, block)
            small = True
        elif op == "attend8":
            n = rng.choice((1, 1, 2, 4, 5, 8, 9, 33, 64, 257, 1100))
            ctx = n + _log_int(rng, 1, 32000)
            window = rng.choice((0, 0, _log_int(rng, 16, 4096)))
            case = _attend8("", B, n, hq, hkv, d, dtype, ctx, page, block, window, rng.choice((0, 4, 16)) if window else 0,
                            1 < n <= 64 and rng.random() < 0.3)
            small = B * ctx * hkv * d <= 1.3e9 and B * n * ctx * hq <= 1.2e9
        elif op == "process":
            rows = rng.choice((1, 2, 5, 8, 9, 17, 33, 65))
            case = _process("", _log_int(rng, 1, 256), rows, rng.choice(VOCABS) + rng.choice((0, 0, 1, 5)),
                            rng.choice(("bf16", "fp32")), _log_int(rng, 1, 16000), rng.choice((0, 0, 1, 20, 300)),
                            rng.random() < 0.4, 1 < rows and rng.random() < 0.4)
            small = True
        else:
            # (generated tokens are counted from nothing here, so that another pass gives the same)
            prompt = rng.random() < 0.7
            case = _count("", _log_int(rng, 1, 256), _log_int(rng, 1, 16000), rng.choice(VOCABS), prompt,
                          not prompt or rng.random() < 0.4)
            small = True
        del case["name"]
        if small and _cost(case) <= limit:
            return case


# ---- inputs -------------------------------------------------------------------------------

def _lengths(case):
    """The sequences' lengths: one sequence has the whole length, several spread from a
    quarter of it (or the new tokens alone) up to it."""
    B, n, ctx = case["B"], case["n"], case["ctx"]
    if B == 1:
        return [ctx]
    lo = max(n, ctx // 4)
    return [lo + (ctx - lo) * b // (B - 1) for b in range(B)]


def _rand(gen, *shape, dtype=torch.float32, std=1.0):
    x = torch.empty(*shape, device="cuda", dtype=dtype)
    return x.normal_(0.0, std, generator=gen)


def _parents(n, gen):
    """A random candidate tree of n nodes, parents before children (-1: the root)."""
    r = torch.rand(n, generator=gen, device="cuda").cpu()
    return [-1] + [int(r[i] * (i + 1)) - 1 for i in range(1, n)]


def _tree_mask(parents):
    n = len(parents)
    mask = torch.eye(n, dtype=torch.uint8)
    depth = [0] * n
    for i, p in enumerate(parents):
        if p >= 0:
            mask[i] |= mask[p]
            depth[i] = depth[p] + 1
    return mask, depth


def _codes(gen, *shape):
    """E4M3 codes as a block's largest value gives them: normal values, the largest near 448."""
    return (_rand(gen, *shape, dtype=torch.float16, std=100.0).clamp_(-E4M3_MAX, E4M3_MAX)).to(torch.float8_e4m3fn)


def _tokens(gen, V, *shape):
    """Token ids of a text: small ids are common, and many come again."""
    return (torch.rand(*shape, generator=gen, device="cuda").double() ** 3 * V).to(torch.int32).clamp_(0, V - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 29)
    dtype = DTYPES.get(case.get("dtype"))
    B = case["B"]
    st = {"case": dict(case)}
    if case["op"] in ("append8", "attend8"):
        n, hkv, d, page, block = case["n"], case["hkv"], case["d"], case["page"], case["block"]
        lens = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        lens = lens[torch.randperm(B, generator=gen, device="cuda")].contiguous()
        per = -(-case["ctx"] // page)
        pages = B * per
        st.update(context_len=lens, k_scale=0.5, v_scale=0.25,
                  block_table=torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(B, per))
        for c in "kv":
            st[c + "_pages"] = _codes(gen, pages, page, hkv, d)
            # scale bytes of 2^-8 to 2^-5: values up to 1.75 to 14 before the tensor's scale
            st[c + "_scales"] = torch.randint(119, 123, (pages, page // block, hkv), generator=gen, device="cuda",
                                              dtype=torch.uint8)
        if case["op"] == "append8":
            # some blocks' new tokens are larger than what the block holds, others smaller
            size = 2.0 ** torch.randint(-3, 3, (B, 1, hkv, 1), generator=gen, device="cuda")
            st.update(k=(_rand(gen, B, n, hkv, d) * size).to(dtype), v=(_rand(gen, B, n, hkv, d) * size).to(dtype),
                      back=n + block - 1, back_len=lens.clamp(max=n + block - 1))
        else:
            st.update(q=_rand(gen, B, n, case["hq"], d, dtype=dtype), scale=1.0 / math.sqrt(d))
            st["tree_mask"] = st["depth"] = None
            if case["tree"]:
                mask, depth = _tree_mask(_parents(n, gen))
                st["tree_mask"], st["depth"] = mask.cuda(), torch.tensor(depth, dtype=torch.int32).cuda()
    elif case["op"] == "process":
        rows, V = case["rows"], case["V"]
        st["logits"] = _rand(gen, B, rows, V, dtype=dtype, std=4.0)
        # half of the history is the prompt
        text = _tokens(gen, V, B, case["history"]).long()
        half = case["history"] // 2
        counts = torch.zeros(B, V, dtype=torch.int32, device="cuda")
        counts.scatter_add_(1, text[:, half:], torch.ones_like(text[:, half:], dtype=torch.int32))
        prompt = torch.zeros(B, V, dtype=torch.bool, device="cuda").scatter_(1, text[:, :half], True)
        st["counts"] = torch.where(prompt, counts + PROMPT, counts)
        # drafts that are in the history, drafts that are not, and one that comes twice
        st["tokens"] = _tokens(gen, V, B, rows - 1) if rows > 1 else None
        st["parents"] = None
        if rows > 2:
            st["tokens"][:, -1] = st["tokens"][:, 0]
        if case["tree"]:
            st["parents"] = torch.tensor(_parents(rows - 1, gen), dtype=torch.int32).cuda()
        st["repetition"] = 1.0 + torch.rand(B, generator=gen, device="cuda") * 0.4
        st["presence"] = torch.rand(B, generator=gen, device="cuda") - 0.3
        st["frequency"] = torch.rand(B, generator=gen, device="cuda") * 0.5
        st["bias_tokens"] = st["bias_values"] = st["mask"] = None
        if case["bias"]:
            k = min(case["bias"], V)
            st["bias_tokens"] = torch.rand(B, V, generator=gen, device="cuda").topk(k, 1).indices.to(torch.int32)
            st["bias_values"] = _rand(gen, B, k, std=5.0)
        if case["mask"]:
            # every other row's grammar leaves few tokens, the others' about half
            words = -(-V // 32)
            m = torch.randint(-2 ** 31, 2 ** 31, (B, rows, words), generator=gen, device="cuda").to(torch.int32)
            few = torch.randint(0, 40, (B, rows, words), generator=gen, device="cuda") == 0
            m[:, ::2] = torch.where(few, m, torch.zeros_like(m))[:, ::2]
            st["mask"] = m
    else:
        st["tokens"] = _tokens(gen, case["V"], B, case["n"])
        st["num_tokens"] = torch.randint(case["n"] // 2, case["n"] + 1, (B,), generator=gen, device="cuda").to(torch.int32)
        if B > 1:
            st["num_tokens"][0] = case["n"]
        # what an earlier request left, or what the request's generated tokens and earlier chunks are
        st["counts"] = (torch.rand(B, case["V"], generator=gen, device="cuda") * 1.1).to(torch.int32)
    return st


# ---- the plain form -----------------------------------------------------------------------

def _slots(st, pos):
    """(page, offset) of logical slots pos [B, S]; slots past the table stand for slot 0."""
    page = st["case"]["page"]
    pos = pos.clamp(0, st["block_table"].shape[1] * page - 1)
    return st["block_table"].long().gather(1, pos // page), pos % page


def _power(e):
    """2^e in 32 bits from its own bits: not by a function that rounds, for products with it meet ties."""
    return ((e + 127) << 23).view(torch.float32)


def _stored(st, c, at):
    """The values in 32 bits that the pages hold at (page, offset), before the tensor's scale."""
    e = st[c + "_scales"][at[0], at[1] // st["case"]["block"]].int() - 127
    return st[c + "_pages"][at].float() * _power(e)[..., None]


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e: 448 is 1.75 * 2^8."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    return torch.where(amax > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, LEAST)).clamp(LEAST, MOST)


def _plain_append8(st):
    c = st["case"]
    n, block, page = c["n"], c["block"], c["page"]
    dev = st["k"].device
    first = st["context_len"].long() - n                               # [B]
    base = first // block * block
    count = (n + block - 2) // block + 1                               # blocks that the new tokens may touch
    slots = base[:, None] + torch.arange(count * block, device=dev)    # [B, count * block]
    new = (slots >= first[:, None]) & (slots < st["context_len"].long()[:, None])
    old = slots < first[:, None]
    i = (slots - first[:, None]).clamp(0, n - 1)
    at = _slots(st, slots)
    rows = torch.arange(c["B"], device=dev)[:, None]
    some = new.view(c["B"], count, block).any(-1)                      # blocks with a new token
    held = old.view(c["B"], count, block).any(-1)
    out = {}
    for w in "kv":
        y = st[w][rows, i].float() * (1.0 / st[w + "_scale"])          # [B, S, hkv, d]
        amax = torch.where(new[..., None], y.abs().amax(-1), torch.zeros((), device=dev))
        e = _exponent(amax.view(c["B"], count, block, c["hkv"]).amax(2))
        blocks = (at[0].view(c["B"], count, block)[..., 0], at[1].view(c["B"], count, block)[..., 0] // block)
        before = st[w + "_scales"][blocks].int() - 127
        e = torch.where(held[..., None], torch.maximum(e, before), e)
        per_slot = e.repeat_interleave(block, 1)
        y = torch.where(old[..., None, None], _stored(st, w, at), y)
        y = (y * _power(-per_slot)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        write = new | old
        st[w + "_pages"].view(torch.uint8)[at[0][write], at[1][write]] = y.view(torch.uint8)[write]
        st[w + "_scales"][blocks[0][some], blocks[1][some]] = (e + 127).to(torch.uint8)[some]
        # read back: the new tokens, and those before them in their first block
        m = st["back"]
        pos = st["context_len"].long()[:, None] - st["back_len"].long()[:, None] + torch.arange(m, device=dev)
        there = torch.arange(m, device=dev) < st["back_len"][:, None]
        v = _stored(st, w, _slots(st, pos)) * st[w + "_scale"]
        out[w] = torch.where(there[..., None, None], v, torch.zeros((), device=dev)).to(st[w].dtype)
    return out


def _plain_attend8(st):
    c = st["case"]
    B, n, hq, hkv, d, window, sinks = (c[k] for k in ("B", "n", "hq", "hkv", "d", "window", "sinks"))
    dev = st["q"].device
    first = st["context_len"].long()[:, None] - n                       # [B, 1]
    new = torch.arange(n, device=dev)
    qpos = first + (new if st["depth"] is None else st["depth"].long())  # [B, n]
    # the slots that some query may see: all, or the first ones and those that end at the length
    if window and window + n + sinks < c["ctx"]:
        tail = st["context_len"].long()[:, None] - (window + n - 1) + torch.arange(window + n - 1, device=dev)
        head = torch.arange(sinks, device=dev).expand(B, sinks)
        slots = torch.cat((head, tail), 1)
        there = torch.cat((head < tail[:, :1].clamp(min=0), tail >= 0), 1)
    else:
        slots = torch.arange(c["ctx"], device=dev).expand(B, c["ctx"])
        there = torch.ones_like(slots, dtype=torch.bool)
    j = slots - first                                                    # index among the new tokens
    kpos = slots if st["depth"] is None else torch.where(j >= 0, first + st["depth"].long()[j.clamp(0, n - 1)], slots)
    if st["tree_mask"] is None:
        sees = j[:, None, :] <= new[:, None]
    else:
        sees = (j < 0)[:, None, :] | (st["tree_mask"].bool()[:, j.clamp(0, n - 1)].transpose(0, 1) & (j < n)[:, None, :])
    sees = sees & there[:, None, :]
    if window:
        sees = sees & ((qpos[:, :, None] - kpos[:, None, :] < window) | (kpos < sinks)[:, None, :])
    at = _slots(st, slots)
    k, v = _stored(st, "k", at), _stored(st, "v", at) * st["v_scale"]
    g = hq // hkv
    q = st["q"].float().view(B, n, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * g, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * (st["scale"] * st["k_scale"])  # [B, hkv, n*g, S]
    s = s.view(B, hkv, n, g, -1).masked_fill_(~sees[:, None, :, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (s - m).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (m + z.log()).squeeze(-1)                                      # [B, hkv, n, g]
    o = torch.matmul(p.view(B, hkv, n * g, -1), v.transpose(1, 2)).view(B, hkv, n, g, d)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, n, hq, d).to(st["q"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, n, hq)}


def _plain_process(st):
    c = st["case"]
    B, rows, V = c["B"], c["rows"], c["V"]
    dev = st["logits"].device
    prompt = st["counts"] < 0
    base = st["counts"] & 0x7FFFFFFF
    if rows > 1:
        if st["parents"] is None:
            sees = torch.ones(rows, rows - 1, device=dev).tril(-1).bool()
        else:
            sees = torch.zeros(rows, rows - 1, dtype=torch.bool)
            for i, p in enumerate(st["parents"].tolist()):
                sees[1 + i] = sees[1 + p]
                sees[1 + i, i] = True
            sees = sees.to(dev)
    bias = None
    if st["bias_tokens"] is not None:
        bias = torch.zeros(B, V, device=dev).scatter_(1, st["bias_tokens"].long(), st["bias_values"])
    r, f, p = (st[k][:, None] for k in ("repetition", "frequency", "presence"))
    bit = torch.arange(V, device=dev)
    out = torch.empty_like(st["logits"])
    for i in range(rows):
        n = base
        if rows > 1:
            n = base.clone().scatter_add_(1, st["tokens"].long(), sees[i].int().expand(B, -1).contiguous())
        x = st["logits"][:, i].float()
        x = torch.where(prompt | (n > 0), torch.where(x > 0, x / r, x * r), x)
        x = x - f * n.float() - p * (n > 0).float()
        if bias is not None:
            x = x + bias
        if st["mask"] is not None:
            allowed = (st["mask"][:, i, bit // 32] >> (bit % 32).int()) & 1
            x = torch.where(allowed > 0, x, torch.full_like(x, -math.inf))
        out[:, i] = x.to(out.dtype)
    return {"logits": out}


def _plain_count(st):
    there = torch.arange(st["case"]["n"], device="cuda") < st["num_tokens"][:, None]
    seen = torch.zeros(st["counts"].shape, dtype=torch.int32, device="cuda")
    seen.scatter_add_(1, st["tokens"].long(), there.int())
    if st["case"]["reset"]:
        st["counts"].zero_()
    if st["case"]["prompt"]:
        st["counts"].copy_(torch.where(seen > 0, st["counts"] | PROMPT, st["counts"]))
    else:
        st["counts"].add_(seen)
    return {"counts": st["counts"]}


# ---- one pass -----------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if not own:
        return {"append8": _plain_append8, "attend8": _plain_attend8, "process": _plain_process, "count": _plain_count}[op](st)
    import speculative_decoding_token_temperature_gb300 as sd
    if op == "process":
        r = sd.process_logits(st["logits"], tokens=st["tokens"], parents=st["parents"], counts=st["counts"],
                              repetition=st["repetition"], presence=st["presence"], frequency=st["frequency"],
                              bias_tokens=st["bias_tokens"], bias_values=st["bias_values"], mask=st["mask"])
        return {"logits": r["logits"]}
    if op == "count":
        sd.count_tokens(st["counts"], st["tokens"], num_tokens=st["num_tokens"], prompt=st["case"]["prompt"], reset=st["case"]["reset"])
        return {"counts": st["counts"]}
    scales = {k: st[k] for k in ("k_scales", "v_scales", "k_scale", "v_scale")}
    if op == "append8":
        sd.append_kv8(st["k"], st["v"], st["k_pages"], st["v_pages"], st["block_table"], st["context_len"], **scales)
        r = sd.read_kv8(st["k_pages"], st["v_pages"], st["block_table"], st["context_len"], st["back"],
                        query_len=st["back_len"], dtype=st["k"].dtype, **scales)
        return {"k": r["k"], "v": r["v"]}
    r = sd.attend(st["q"], st["k_pages"], st["v_pages"], st["block_table"], st["context_len"],
                  tree_mask=st["tree_mask"], depth=st["depth"], window=st["case"]["window"],
                  sinks=st["case"]["sinks"], scale=st["scale"], with_lse=True, **scales)
    return {"out": r["out"], "lse": r["lse"]}


# ---- what a pass cannot do without --------------------------------------------------------

def _visible(case):
    """(cache slots that some query sees, scales of their blocks, pairs of a query token and a slot
    it sees), summed over the sequences.  A tree's pairs among its own nodes count as half of all pairs."""
    n, w, sinks, block = case["n"], case["window"], case["sinks"], case["block"]
    slots = blocks = pairs = 0
    for L in _lengths(case):
        P = L - n
        lo = max(0, P + 1 - w) if w else 0
        here = L if lo <= sinks else L - lo + sinks
        slots += here
        blocks += -(-here // block)
        if not w:
            pairs += n * P + n * (n + 1) // 2
            continue
        for i in range(n):
            pos = P + i
            lo = max(0, pos + 1 - w)
            pairs += pos + 1 - lo + min(sinks, lo)
    return slots, blocks, pairs


def work(case):
    B = case["B"]
    if case["op"] == "append8":
        n, hkv, d, block = case["n"], case["hkv"], case["d"], case["block"]
        new = B * n * hkv * d
        back = sum(min(L, n + block - 1) for L in _lengths(case)) * hkv * d
        # the 16-bit values in, codes out; the codes that are read back in, and their values out
        return {"bytes": 2 * (new * 3 + back * 3) + 2 * B * hkv * (n // block + 1), "flops": 8 * new + 4 * back}
    if case["op"] == "attend8":
        n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
        slots, blocks, pairs = _visible(case)
        return {"bytes": 2 * hkv * (slots * d + blocks) + 2 * 2 * B * n * hq * d + 4 * B * n * hq, "flops": 4 * pairs * hq * d}
    if case["op"] == "process":
        rows, V = case["rows"], case["V"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": B * rows * V * 2 * size + 4 * B * V + 8 * B * case["bias"] + (B * rows * (-(-V // 32)) * 4 if case["mask"] else 0),
                "flops": 5 * B * rows * V}
    # a table from nothing is written whole; more of a prompt touches its own tokens
    tokens = B * case["n"]
    return {"bytes": 4 * tokens + (4 * B * case["V"] if case["reset"] else 8 * tokens), "flops": tokens}


# ---- the definitions in 64 bits -----------------------------------------------------------

def _e4m3_table():
    """The value of every E4M3 byte (127 and 255 are NaN)."""
    v = [m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    v[127] = math.nan
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device="cuda")


def _power64(e):
    """2^e of whole exponents, from a table: quotients by it meet ties."""
    return torch.tensor([2.0 ** i for i in range(-128, 129)], dtype=torch.float64, device="cuda")[e.long() + 128]


def _nearest_e4m3(t):
    """The nearest E4M3 value of each t, ties to the even code, saturated."""
    grid = _e4m3_table()[:127]
    a = t.abs().clamp(max=E4M3_MAX)
    up = torch.searchsorted(grid, a).clamp(1, 126)
    below, above = a - grid[up - 1], grid[up] - a
    pick = torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)
    return grid[pick] * t.sign()


def _exact_append8(st):
    """One block at a time along a sequence; rounding to 8 bits is part of the definition (the product
    with 1 / the tensor's scale in 32 bits, as the definition has it)."""
    c = st["case"]
    n, block, page, hkv, d = c["n"], c["block"], c["page"], c["hkv"], c["d"]
    table = _e4m3_table()
    out = {}
    for w in "kv":
        res = torch.zeros(c["B"], st["back"], hkv, d, dtype=torch.float64, device="cuda")
        for b, L in enumerate(st["context_len"].tolist()):
            first, m = L - n, min(L, st["back"])
            start = first // block * block
            values = torch.zeros(L - start, hkv, d, dtype=torch.float64, device="cuda")
            blocks = -(-(L - start) // block)
            pg = st["block_table"][b].long()
            y = (st[w][b].float() * (1.0 / st[w + "_scale"])).double()
            values[first - start:] = y
            # the smallest power of two, for every block and head
            padded = torch.zeros(blocks * block, hkv, d, dtype=torch.float64, device="cuda")
            padded[first - start:L - start] = y.abs()
            amax = padded.view(blocks, block, hkv, d).amax((1, 3))
            powers = E4M3_MAX * _power64(torch.arange(LEAST, MOST + 1, device="cuda"))
            e = torch.searchsorted(powers, amax).clamp(max=MOST - LEAST) + LEAST
            if first > start:
                s = torch.arange(start, first, device="cuda")
                before = st[w + "_scales"][pg[start // page], start % page // block].long() - 127
                kept = table[st[w + "_pages"].view(torch.uint8)[pg[s // page], s % page].long()] * _power64(before)[:, None]
                values[:first - start] = kept
                e[0] = torch.maximum(e[0], before)
            scale = _power64(e).repeat_interleave(block, 0)[:L - start, :, None]
            values = _nearest_e4m3(values / scale) * scale * st[w + "_scale"]
            # tokens before the first block that is written are as they were
            s = torch.arange(L - m, start, device="cuda")
            if len(s):
                e0 = st[w + "_scales"][pg[s // page], s % page // block].long() - 127
                kept = table[st[w + "_pages"].view(torch.uint8)[pg[s // page], s % page].long()] * _power64(e0)[..., None]
                values = torch.cat((kept * st[w + "_scale"], values))
            res[b, :m] = values[len(values) - m:]
        out[w] = res
    return out


def _exact_attend8(st):
    c = st["case"]
    n, hq, hkv, d, page, block = c["n"], c["hq"], c["hkv"], c["d"], c["page"], c["block"]
    out = torch.zeros(c["B"], n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], n, hq), -math.inf, dtype=torch.float64, device="cuda")
    table = _e4m3_table()

    def cached(which, pg, off):
        x = table[st[which + "_pages"].view(torch.uint8)[pg, off].int()]
        s = _power64(st[which + "_scales"][pg, off // block].long() - 127)
        return x * s[..., None] * st[which + "_scale"]

    heads = torch.arange(hq, device="cuda") // (hq // hkv)
    for b, L in enumerate(st["context_len"].tolist()):
        P = L - n
        depth = torch.arange(n, device="cuda") if st["depth"] is None else st["depth"].long()
        position = torch.cat((torch.arange(P, device="cuda"), P + depth))
        allowed = torch.ones(n, L, dtype=torch.bool, device="cuda")
        allowed[:, P:] = torch.ones(n, n, device="cuda").tril().bool() if st["tree_mask"] is None else st["tree_mask"].bool()
        if c["window"]:
            near = position[None, :] > (position[P:] - c["window"])[:, None]
            allowed &= near | (position < c["sinks"])[None, :]
        kept = allowed.any(0).nonzero().squeeze(-1)
        if not len(kept):
            continue
        allowed = allowed[:, kept]
        pg, off = st["block_table"][b].long()[kept // page], kept % page
        k, v = cached("k", pg, off), cached("v", pg, off)
        for h in range(hkv):
            mine = (heads == h).nonzero().squeeze(-1)
            s = torch.einsum("ngd,sd->ngs", st["q"][b][:, mine].double(), k[:, h]) * st["scale"]
            s = torch.where(allowed[:, None, :], s, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            z = torch.logsumexp(s, -1)
            lse[b][:, mine] = z
            w = torch.where(z[..., None] > -math.inf, torch.exp(s - z[..., None]), torch.zeros_like(s))
            out[b][:, mine] = torch.einsum("ngs,sd->ngd", w, v[:, h])
    return {"out": out, "lse": lse}


def _exact_process(st):
    """One sequence at a time: its counts for every row by a histogram of the row's own drafts."""
    c = st["case"]
    B, rows, V = c["B"], c["rows"], c["V"]
    out = torch.empty(B, rows, V, dtype=torch.float64, device="cuda")
    paths = [[]]
    for i in range(rows - 1):
        parent = i - 1 if st["parents"] is None else int(st["parents"][i])
        paths.append(paths[1 + parent] + [i])
    at = torch.tensor([(i, j) for i, path in enumerate(paths) for j in path], dtype=torch.long, device="cuda").view(-1, 2)
    for b in range(B):
        x = st["logits"][b].double()
        counts = st["counts"][b].long()
        prompt = counts < 0
        n = (counts + prompt.long() * 2 ** 31).expand(rows, V).double().clone()
        if len(at):
            n.index_put_((at[:, 0], st["tokens"][b].long()[at[:, 1]]), torch.ones(len(at), dtype=torch.float64, device="cuda"),
                         accumulate=True)
        r, p, f = (st[k][b].double() for k in ("repetition", "presence", "frequency"))
        factor = torch.where(x > 0, 1 / r, r)
        x = torch.where((n > 0) | prompt, x * factor, x) - n * f - (n > 0) * p
        if st["bias_tokens"] is not None:
            x[:, st["bias_tokens"][b].long()] += st["bias_values"][b].double()
        if st["mask"] is not None:
            words = st["mask"][b].long() & 0xFFFFFFFF
            bits = (words[..., None] // (2 ** torch.arange(32, device="cuda")) % 2).reshape(rows, -1)[:, :V]
            x[bits == 0] = -math.inf
        out[b] = x
    return {"logits": out}


def exact(case, seed):
    if case["op"] == "count":
        return None  # whole numbers
    st = prepare(case, seed)
    return {"append8": _exact_append8, "attend8": _exact_attend8, "process": _exact_process}[case["op"]](st)
