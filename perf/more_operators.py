"""Cases of the decode step's other operators: what a request's rules do to
logits before a token is drawn (adjust_logits), new keys and values written
into the pages of a paged cache with the position rotation on the way
(pages_append), and attention over such a cache held in 8 bits (pages_attend).

`own` False runs the plain form in elementary torch operations, `own` True
the library's calls.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
LOWEST = -100  # the least exponent of a block's scale


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _adjust(name, rows, vocab, dtype, history, biases, mask):
    return {"name": name, "op": "adjust", "rows": rows, "vocab": vocab, "dtype": dtype, "history": history,
            "biases": biases, "mask": mask}


def _append(name, rows, tokens, past, heads, q_heads, dim, rotated, interleaved, page_tokens, block_tokens, dtype, cache):
    return {"name": name, "op": "append", "rows": rows, "tokens": tokens, "past": past, "heads": heads,
            "q_heads": q_heads, "dim": dim, "rotated": rotated, "interleaved": interleaved,
            "page_tokens": page_tokens, "block_tokens": block_tokens, "dtype": dtype, "cache": cache}


def _attend(name, rows, length, ragged, drafts, heads, group, dim, page_tokens, block_tokens, dtype):
    return {"name": name, "op": "attend", "rows": rows, "length": length, "ragged": ragged, "drafts": drafts,
            "heads": heads, "group": group, "dim": dim, "page_tokens": page_tokens, "block_tokens": block_tokens,
            "dtype": dtype}


def listed():
    return [
        # one user's next token after a short chat, all three penalties: latency alone
        _adjust("adjust_one_row", 1, 32000, "bf16", 200, 0, False),
        # a few requests that set everything, an odd vocabulary, a grammar's mask, a handful of biases
        _adjust("adjust_mixed_odd", 7, 50257, "f32", 1000, 5, True),
        # a batch of long conversations: as much history as a quarter of the vocabulary
        _adjust("adjust_long_history", 48, 131072, "bf16", 32768, 0, False),
        # the largest decode batch and vocabulary, masks and the longest lists of biases, more than L2 holds
        _adjust("adjust_large", 256, 262144, "f32", 2048, 300, True),
        # a server's decode step: one token a row into the 8-bit cache, queries rotated with it
        _append("append_step", 64, 64, 2000, 8, 32, 128, 128, False, 16, 16, "bf16", "e4m3"),
        # one user's next token into a cache of the model's own type
        _append("append_one", 1, 1, 1000, 8, 32, 128, 128, False, 16, 16, "bf16", "bf16"),
        # chunks of a few prompts at once, ragged, many query heads
        _append("append_prompts", 5, 8192, 500, 8, 64, 128, 128, False, 16, 16, "bf16", "bf16"),
        # a long prompt's chunk into the 8-bit cache: interleaved pairs, half of a head rotated, odd pages
        _append("append_prompts_8bit", 9, 16384, 300, 16, 16, 64, 32, True, 48, 24, "f16", "e4m3"),
        # one user's next token after some pages of text: latency alone
        _attend("attend_one_row", 1, 4000, False, 1, 8, 4, 128, 16, 16, "bf16"),
        # drafts of a few tokens to be verified, seven query heads a key head, pages that no tile divides
        _attend("attend_drafts", 33, 3001, True, 5, 4, 7, 64, 20, 10, "f16"),
        # a server's decode batch of ragged rows, more than L2 holds
        _attend("attend_batch", 64, 8192, True, 1, 8, 8, 128, 16, 16, "bf16"),
        # two users' very long contexts: the rows are few and the axis is long
        _attend("attend_long", 2, 200000, False, 1, 8, 8, 128, 64, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["adjust", "append", "attend"])
    if op == "adjust":
        dtype = rng.choice(["bf16", "f16", "f32"])
        vocab = _log(rng, 1000, 262144)
        rows = _log(rng, 1, max(1, min(256, (64 << 20) // vocab)))
        history = _log(rng, 1, max(1, min(32768, (2 << 20) // rows)))
        return _adjust("", rows, vocab, dtype, history, rng.choice([0, 0, 3, 30, 300]), rng.random() < 0.5)
    dtype = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    heads = rng.choice([1, 2, 4, 8, 8, 16])
    group = rng.choice([1, 2, 3, 4, 4, 7, 8, 8, 16])
    block_tokens = rng.choice([1, 8, 10, 16, 16, 16, 24, 64])
    page_tokens = block_tokens * rng.choice([1, 1, 2, 4])
    if op == "append":
        q_heads = min(64, heads * group)
        tokens = _log(rng, 1, max(1, min(16384, (96 << 20) // (dim * (q_heads + 2 * heads)))))
        rows = tokens if rng.random() < 0.4 and tokens <= 256 else min(tokens, _log(rng, 1, 32))
        return _append("", rows, tokens, _log(rng, 4, 2000), heads, q_heads, dim, rng.choice([dim, dim, dim // 2]),
                       rng.random() < 0.4, page_tokens, block_tokens, dtype, rng.choice([dtype, "e4m3", "e4m3"]))
    rows = _log(rng, 1, 256)
    length = _log(rng, 16, max(64, min(200000, (380 << 20) // (rows * heads * dim))))
    drafts = rng.choice([1, 1, 1, 2, 5, 8])
    return _attend("", rows, length, rng.random() < 0.7, drafts, heads, group, dim, page_tokens, block_tokens, dtype)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)


def _uniform(g, n):
    return torch.rand(n, generator=g, device=DEV)


def _pick(g, n, values, dtype):
    idx = torch.randint(len(values), (n,), generator=g, device=DEV)
    return torch.tensor(values, dtype=dtype, device=DEV)[idx]


def _prepare_adjust(c, g):
    rows, vocab, dtype = c["rows"], c["vocab"], DTYPES[c["dtype"]]
    logits = torch.randn(rows, vocab, generator=g, device=DEV).mul_(2.5).to(dtype)
    st = {"logits": logits, "out": torch.empty_like(logits)}
    # text repeats itself: most tokens come from the small end of the vocabulary
    h = c["history"]
    st["history"] = (_uniform(g, rows * h).pow(3) * vocab).to(torch.int32).clamp_(max=vocab - 1).view(rows, h)
    st["history_lens"] = (h * (1 - 0.6 * _uniform(g, rows))).ceil().to(torch.int32)
    st["prompt_lens"] = (st["history_lens"] * _uniform(g, rows)).to(torch.int32)
    st["repetition"] = _pick(g, rows, [1.0, 1.05, 1.1, 1.3], torch.float32)
    st["presence"] = _pick(g, rows, [0.0, 0.1, 0.6], torch.float32)
    st["frequency"] = _pick(g, rows, [0.0, 0.05, 0.3], torch.float32)
    st["bias_tokens"] = st["bias"] = st["allowed"] = None
    if c["biases"]:
        n = min(c["biases"], vocab // 2)
        # distinct tokens in any order: one out of each of n equal parts of the vocabulary
        at = (torch.arange(n, device=DEV) * (vocab // n)) + (_uniform(g, rows * n).view(rows, n) * (vocab // n)).long()
        at = torch.gather(at, 1, torch.argsort(_uniform(g, rows * n).view(rows, n), 1))
        st["bias_tokens"] = at.to(torch.int32).contiguous()
        st["bias"] = _pick(g, rows * n, [-100.0, -2.0, 1.5, 5.0], torch.float32).view(rows, n)
    if c["mask"]:
        words = (vocab + 31) // 32
        keep = _uniform(g, rows)[:, None].pow(3)  # the share of the vocabulary a row's grammar allows
        bits = torch.rand(rows, words * 32, generator=g, device=DEV) < keep
        shift = torch.arange(32, device=DEV)
        packed = torch.empty(rows, words, dtype=torch.int64, device=DEV)
        for r in range(0, rows, 64):
            packed[r : r + 64] = (bits[r : r + 64].view(-1, words, 32).long() << shift).sum(2)
        st["allowed"] = torch.where(packed >= 2**31, packed - 2**32, packed).to(torch.int32)
    return st


def _spread(g, n, most, power=1):
    """n numbers up to `most`, the same ones for every seed, in an order of the seed's own."""
    share = (torch.arange(n, 0, -1, dtype=torch.float64, device=DEV) / n).pow(power)
    return (share * most).long()[torch.randperm(n, generator=g, device=DEV)]


def _pages(g, counts, page_tokens, tokens):
    """A table of randomly placed pages for rows of `counts` tokens, `tokens` in all at most, and the
    number of pages; some are free."""
    n = (counts + page_tokens - 1) // page_tokens
    width, total = int(n.max()), int(n.sum())
    pages = tokens // page_tokens + counts.numel() + 1
    place = torch.randperm(pages, generator=g, device=DEV)
    table = torch.full((counts.numel(), width), -1, dtype=torch.int64, device=DEV)
    table[torch.arange(width, device=DEV)[None, :] < n[:, None]] = place[:total]
    return table.to(torch.int32), pages


def _cache(g, pages, c):
    """Keys, values and, for the 8-bit cache, the scales of their blocks."""
    shape = (pages, c["page_tokens"], c["heads"], c["dim"])
    dtype = DTYPES[c.get("cache", "e4m3")]
    made = []
    for _ in range(2):
        t = torch.empty(shape, dtype=dtype, device=DEV)
        step = max(1, (1 << 27) // max(1, shape[1] * shape[2] * shape[3]))
        for p in range(0, pages, step):
            x = torch.randn(min(step, pages - p), *shape[1:], generator=g, device=DEV)
            t[p : p + step] = (x.mul_(110.0).clamp_(-448.0, 448.0) if dtype is DTYPES["e4m3"] else x).to(dtype)
        made.append(t)
    if dtype is not DTYPES["e4m3"]:
        return (*made, None, None)
    blocks = c["page_tokens"] // c["block_tokens"]
    for _ in range(2):
        e = torch.randint(-8, -5, (pages, blocks, c["heads"]), generator=g, device=DEV)
        made.append(torch.exp2(e.double()).float())
    return made


def _hold(st, keys, values, key_scales, value_scales):
    st["keys"], st["values"], st["key_scales"], st["value_scales"] = keys, values, key_scales, value_scales
    if own:  # a program makes it once for a cache
        import u32_prefix_scan_gb300 as u

        st["cache"] = u.KVCache(keys, values, key_scales, value_scales)


def _starts(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _prepare_append(c, g):
    rows, tokens, dim, pt = c["rows"], c["tokens"], c["dim"], c["page_tokens"]
    dtype = DTYPES[c["dtype"]]
    # every row has a token at least, some have many
    counts = 1 + _spread(g, rows, 1 << 20, 2) * (tokens - rows) // int(_spread(g, rows, 1 << 20, 2).sum())
    counts[0] += tokens - counts.sum()
    past = _spread(g, rows, c["past"])
    lens = past + counts
    st = {"counts": counts, "lens": lens.to(torch.int32), "starts": None if rows == tokens else _starts(counts)}
    st["table"], pages = _pages(g, lens, pt, rows * c["past"] + tokens)
    _hold(st, *_cache(g, pages, c))
    # one projection gives queries, keys and values side by side
    heads, q_heads = c["heads"], c["q_heads"]
    qkv = torch.randn(tokens, (q_heads + 2 * heads) * dim, generator=g, device=DEV)
    qkv *= torch.exp2(torch.randint(-2, 3, (tokens, 1), generator=g, device=DEV).float())
    qkv = qkv.to(dtype).view(tokens, q_heads + 2 * heads, dim)
    st["queries"], st["new_keys"] = qkv[:, :q_heads], qkv[:, q_heads : q_heads + heads]
    st["new_values"] = qkv[:, q_heads + heads :]
    st["queries_out"] = torch.empty(tokens, q_heads, dim, dtype=dtype, device=DEV)
    half = c["rotated"] // 2
    rate = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    angle = torch.arange(int(lens.max()) + 7, dtype=torch.float64, device=DEV)[:, None] * rate
    st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
    st["interleaved"] = c["interleaved"]
    return st


def _prepare_attend(c, g):
    rows, heads, dim, dtype = c["rows"], c["heads"], c["dim"], DTYPES[c["dtype"]]
    counts = torch.full((rows,), c["drafts"], dtype=torch.int64, device=DEV)
    if c["drafts"] > 1:
        counts = 1 + _spread(g, rows, c["drafts"] - 1)
    lens = torch.full((rows,), c["length"], dtype=torch.int64, device=DEV)
    if c["ragged"]:
        lens = _spread(g, rows, c["length"])
    lens = torch.maximum(lens, counts)
    st = {"lens": lens.to(torch.int32), "starts": None if c["drafts"] == 1 else _starts(counts)}
    st["longest"], st["most"] = int(lens.max()), c["drafts"]
    held = rows * c["length"]
    if c["ragged"]:
        held = rows * (c["length"] + rows + 2 * c["drafts"]) // 2 + c["length"]
    st["table"], pages = _pages(g, lens, c["page_tokens"], held)
    _hold(st, *_cache(g, pages, c))
    tokens = int(counts.sum())
    q = torch.randn(tokens, heads * c["group"], dim, generator=g, device=DEV)
    st["queries"] = (q * _pick(g, tokens, [0.5, 1.0, 3.0], torch.float32)[:, None, None]).to(dtype)
    st["out"] = torch.empty_like(st["queries"])
    st["scale"] = 1.0 / math.sqrt(dim)
    return st


_PREPARE = {"adjust": _prepare_adjust, "append": _prepare_append, "attend": _prepare_attend}


def prepare(case, seed):
    st = _PREPARE[case["op"]](case, _gen(seed))
    st["op"] = case["op"]
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    return _OWN[state["op"]](state) if own else _PLAIN[state["op"]](state)


def _own_adjust(st):
    import u32_prefix_scan_gb300 as u

    return u.adjust_logits(st["logits"], history=st["history"], history_lens=st["history_lens"],
                           prompt_lens=st["prompt_lens"], repetition=st["repetition"], presence=st["presence"],
                           frequency=st["frequency"], bias_tokens=st["bias_tokens"], bias=st["bias"],
                           allowed=st["allowed"], out=st["out"])


def _own_append(st):
    import u32_prefix_scan_gb300 as u

    q = u.pages_append(st["cache"], st["table"], st["lens"], st["new_keys"], st["new_values"], starts=st["starts"],
                       cos=st["cos"], sin=st["sin"], interleaved=st["interleaved"], queries=st["queries"],
                       queries_out=st["queries_out"])
    return [st["keys"], st["values"], q, st["key_scales"], st["value_scales"]]


def _own_attend(st):
    import u32_prefix_scan_gb300 as u

    return u.pages_attend(st["cache"], st["table"], st["lens"], st["queries"], starts=st["starts"], scale=st["scale"],
                          out=st["out"])


_OWN = {"adjust": _own_adjust, "append": _own_append, "attend": _own_attend}


def _plain_adjust(st):
    logits, history = st["logits"], st["history"].long()
    rows, vocab = logits.shape
    x = logits.float()
    at = torch.arange(history.shape[1], device=DEV)[None, :]
    held = at < st["history_lens"][:, None]
    made = held & (at >= st["prompt_lens"][:, None])
    seen = torch.zeros(rows, vocab, dtype=torch.int32, device=DEV).scatter_add_(1, history, held.int()) > 0
    count = torch.zeros(rows, vocab, dtype=torch.int32, device=DEV).scatter_add_(1, history, made.int())
    r = st["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    less = x - st["frequency"][:, None] * count
    x = torch.where(count > 0, less - st["presence"][:, None], x)
    if st["bias"] is not None:
        x = x.scatter_add(1, st["bias_tokens"].long(), st["bias"])
    if st["allowed"] is not None:
        bits = (st["allowed"][:, :, None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        x = x.masked_fill(bits.view(rows, -1)[:, :vocab] == 0, float("-inf"))
    return x.to(logits.dtype)


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, dim] in 32 bits, cos and sin [tokens, pairs]."""
    pairs = cos.shape[1]
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0 : 2 * pairs : 2], x[..., 1 : 2 * pairs : 2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :pairs], x[..., pairs : 2 * pairs]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., 2 * pairs :]], -1)


def _power(e):
    """2^e as float32, by its bits."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantised(cache, scales, table, first, page, slot, x):
    """Writes x [tokens, heads, dim] at (page, slot); `first`: each row's first new position."""
    pages, page_tokens, heads, dim = cache.shape
    blocks = scales.shape[1]
    size = page_tokens // blocks
    flat = scales.view(pages * blocks, heads)
    block = page * blocks + slot // size
    f, e = torch.frexp(x.abs().amax(-1))
    need = torch.where(f == 0, LOWEST, (e - torch.where(f <= 0.875, 9, 8)).clamp(min=LOWEST))
    need = torch.full((pages * blocks, heads), LOWEST, dtype=need.dtype, device=DEV).scatter_reduce_(
        0, block[:, None].expand(-1, heads), need, "amax")
    # a row's first block may hold older tokens: its scale does not fall, and they are told in the new one
    within = torch.arange(size, device=DEV)[None, :]
    p0 = torch.gather(table, 1, (first // page_tokens)[:, None])[:, 0].long()
    b0 = p0 * blocks + first % page_tokens // size
    past = first % size
    old = torch.where((past > 0)[:, None], flat[b0], 0.0)
    scale = torch.maximum(_power(need[b0]), old)
    codes = cache.view(pages * blocks, size, heads, dim)
    held = codes[b0].float()
    told = torch.where((within < past[:, None])[:, :, None, None], held * (old / scale)[:, None, :, None], held)
    codes[b0] = told.to(cache.dtype)
    flat[block] = _power(need[block])
    flat[b0] = scale
    cache[page, slot] = (x * (1.0 / flat[block])[:, :, None]).to(cache.dtype)


def _plain_append(st):
    table, lens, counts = st["table"], st["lens"].long(), st["counts"]
    keys, values = st["keys"], st["values"]
    tokens, page_tokens = st["new_keys"].shape[0], keys.shape[1]
    row = torch.repeat_interleave(torch.arange(counts.numel(), device=DEV), counts, output_size=tokens)
    first = lens - counts
    ends = counts.cumsum(0)
    at = torch.arange(tokens, device=DEV) - (ends - counts)[row] + first[row]
    page, slot = table[row, at // page_tokens].long(), at % page_tokens
    cos, sin = st["cos"][at], st["sin"][at]
    k = _rotate(st["new_keys"].float(), cos, sin, st["interleaved"])
    q = _rotate(st["queries"].float(), cos, sin, st["interleaved"]).to(st["queries"].dtype)
    v = st["new_values"].float()
    if st["key_scales"] is None:
        keys[page, slot], values[page, slot] = k.to(keys.dtype), v.to(values.dtype)
    else:
        _quantised(keys, st["key_scales"], table, first, page, slot, k)
        _quantised(values, st["value_scales"], table, first, page, slot, v)
    return [keys, values, q, st["key_scales"], st["value_scales"]]


def _plain_attend(st):
    keys, values, table, lens = st["keys"], st["values"], st["table"], st["lens"].long()
    pages, page_tokens, heads, dim = keys.shape
    size = page_tokens // st["key_scales"].shape[1]
    rows, longest, most = lens.numel(), st["longest"], st["most"]
    q = st["queries"]
    starts = torch.arange(rows + 1, device=DEV) if st["starts"] is None else st["starts"].long()
    counts = starts[1:] - starts[:-1]
    at = torch.arange(longest, device=DEV)
    page = table[:, at // page_tokens].clamp(min=0).long()
    slot = (at % page_tokens)[None, :].expand(rows, -1)
    k = keys[page, slot].float() * st["key_scales"][page, slot // size][..., None]
    nth = torch.arange(most, device=DEV)
    token = (starts[:-1, None] + nth).clamp(max=q.shape[0] - 1)
    # [rows, heads, drafts * group, dim]
    queries = q[token].float().view(rows, most, heads, -1, dim).permute(0, 2, 1, 3, 4)
    group = queries.shape[3]
    s = queries.reshape(rows, heads, most * group, dim) @ k.permute(0, 2, 3, 1)
    del k
    s = (s * st["scale"]).view(rows, heads, most, group, longest)
    last = (lens - counts)[:, None] + nth  # each query's own position
    hidden = at[None, None, :] > torch.minimum(last, lens[:, None] - 1)[:, :, None]
    s = s.masked_fill(hidden[:, None, :, None, :], float("-inf"))
    s = torch.exp(s - s.amax(-1, keepdim=True))
    s = s / s.sum(-1, keepdim=True)
    v = values[page, slot].float() * st["value_scales"][page, slot // size][..., None]
    o = s.view(rows, heads, most * group, longest) @ v.permute(0, 2, 1, 3)
    o = o.view(rows, heads, most, group, dim).permute(0, 2, 1, 3, 4).reshape(rows * most, heads * group, dim)
    row = torch.searchsorted(starts[1:], torch.arange(q.shape[0], device=DEV), right=True)
    return o[row * most + torch.arange(q.shape[0], device=DEV) - starts[row]].to(q.dtype)


_PLAIN = {"adjust": _plain_adjust, "append": _plain_append, "attend": _plain_attend}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_adjust(c, st):
    made = []
    for r in range(c["rows"]):
        x = st["logits"][r].double()
        n, prompt = int(st["history_lens"][r]), int(st["prompt_lens"][r])
        tokens, _ = st["history"][r, :n].unique(return_counts=True)
        tokens = tokens.long()
        some = x[tokens]
        rep = st["repetition"][r].double()
        x[tokens] = torch.where(some > 0, some / rep, some * rep)
        tokens, counts = st["history"][r, prompt:n].unique(return_counts=True)
        x[tokens.long()] -= counts * st["frequency"][r].double() + st["presence"][r].double()
        if st["bias"] is not None:
            x[st["bias_tokens"][r].long()] += st["bias"][r].double()
        if st["allowed"] is not None:
            i = torch.arange(c["vocab"], device=DEV)
            x[(st["allowed"][r].long()[i // 32] >> (i % 32)) % 2 == 0] = float("-inf")
        made.append(x)
    return torch.stack(made)


def _exact_append(c, st):
    first = st["lens"].long() - st["counts"]
    lists = [st["queries"].double(), st["new_keys"].double(), st["new_values"].double()]
    half, dim = c["rotated"] // 2, c["dim"]
    order = torch.arange(dim, device=DEV)
    a, b = (order[0 : 2 * half : 2], order[1 : 2 * half : 2]) if c["interleaved"] else (order[:half], order[half : 2 * half])
    whole = st["key_scales"] is None  # values that were rounded to 8 bits have no other form
    keys, values = (st["keys"].double(), st["values"].double()) if whole else (None, None)
    q = lists[0].clone()
    begin = 0
    for r, n in enumerate(st["counts"].tolist()):
        at = int(first[r]) + torch.arange(n, device=DEV)
        z = torch.complex(st["cos"][at].double(), st["sin"][at].double())[:, None, :]
        new = lists[1][begin : begin + n].clone()
        for x in (q[begin : begin + n], new):
            y = torch.complex(x[..., a], x[..., b]) * z
            x[..., a], x[..., b] = y.real, y.imag
        if whole:
            where = st["table"][r].long()[at // c["page_tokens"]] * c["page_tokens"] + at % c["page_tokens"]
            keys.view(-1, c["heads"], dim)[where] = new
            values.view(-1, c["heads"], dim)[where] = lists[2][begin : begin + n]
        begin += n
    return [keys, values, q, None, None]


def _exact_attend(c, st):
    size, group = c["block_tokens"], c["group"]
    out = torch.empty(st["queries"].shape, dtype=torch.float64, device=DEV)
    begin = 0
    starts = None if st["starts"] is None else st["starts"].tolist()
    for r, n in enumerate(st["lens"].tolist()):
        new = 1 if starts is None else starts[r + 1] - starts[r]
        used = -(-n // c["page_tokens"])
        pages = st["table"][r, :used].long()
        for h in range(c["heads"]):
            kv = []
            for codes, scales in ((st["keys"], st["key_scales"]), (st["values"], st["value_scales"])):
                s = scales[pages, :, h].double().repeat_interleave(size, 1)
                kv.append((codes[pages, :, h].double() * s[:, :, None]).reshape(-1, c["dim"])[:n])
            for i in range(new):
                seen = n - new + i + 1
                w = st["queries"][begin + i, h * group : (h + 1) * group].double() @ kv[0][:seen].T * st["scale"]
                out[begin + i, h * group : (h + 1) * group] = torch.softmax(w, -1) @ kv[1][:seen]
        begin += new
    return out


_EXACT = {"adjust": _exact_adjust, "append": _exact_append, "attend": _exact_attend}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "adjust":
        logits = c["rows"] * c["vocab"]
        lists = c["rows"] * (0.7 * 4 * c["history"] + 8 * c["biases"])
        return {"bytes": 2 * SIZES[c["dtype"]] * logits + lists + (logits / 8 if c["mask"] else 0),
                "flops": c["rows"] * (3 * 0.7 * c["history"] + c["biases"])}
    if c["op"] == "append":
        new, heads = c["tokens"] * c["dim"], 2 * c["heads"]
        size = SIZES[c["dtype"]]
        angles = 4 * c["rotated"] * min(c["tokens"], c["past"] + c["tokens"])
        scales = 4 * heads * c["tokens"] / c["block_tokens"] if c["cache"] == "e4m3" else 0
        return {"bytes": new * (size * (heads + 2 * c["q_heads"]) + SIZES[c["cache"]] * heads) + angles + scales,
                "flops": 3 * c["tokens"] * c["rotated"] * (c["heads"] + c["q_heads"])}
    held = c["rows"] * c["length"] * (0.5 if c["ragged"] else 1.0)
    queries = c["rows"] * (1 + c["drafts"]) / 2 * c["heads"] * c["group"]
    per_token = 2 * c["heads"] * (c["dim"] + 4 / c["block_tokens"]) + 4 / c["page_tokens"]
    return {"bytes": held * per_token + 2 * SIZES[c["dtype"]] * queries * c["dim"],
            "flops": 4 * c["dim"] * held / c["rows"] * queries}
