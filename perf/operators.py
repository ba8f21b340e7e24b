"""Cases of the decode-step operators: choosing the next token of every row
(sample_tokens) and keeping the pages of a paged cache (pages_copy,
pages_fork, pages_free, pages_compact).

Every operator is exact on integers, so both forms below give the same bits:
`own` False runs the plain form in elementary torch operations, `own` True
the library's calls.
"""

import numpy as np
import torch

own = False

DEV = "cuda"
LOG2E = float(np.float32(1.4426950408889634))
# 2^-f on [-0.5, 0.5] as 1 + f (C1 + f (C2 + ...)), in f32, each operation rounded alone
POLY = [float.fromhex(c) for c in ("-0x1.62e42ap-1", "0x1.ebf9bcp-3", "-0x1.c6b752p-5", "0x1.3cea88p-7",
                                   "-0x1.5bba14p-10")]
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _sample(name, rows, vocab, dtype, mode, mask="none"):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "mode": mode, "mask": mask}


def _copy(name, pages, n, planes, page_bytes):
    return {"name": name, "op": "copy", "pages": pages, "n": n, "planes": planes, "page_bytes": page_bytes}


def _fork(name, rows, width, pages, page_tokens, kids, planes, page_bytes, used=0.8):
    return {"name": name, "op": "fork", "rows": rows, "width": width, "pages": pages, "page_tokens": page_tokens,
            "kids": kids, "used": used, "planes": planes, "page_bytes": page_bytes}


def _free(name, rows, width, pages, page_tokens):
    return {"name": name, "op": "free", "rows": rows, "width": width, "pages": pages, "page_tokens": page_tokens}


def _compact(name, rows, width, pages, page_tokens, live, planes, page_bytes):
    return {"name": name, "op": "compact", "rows": rows, "width": width, "pages": pages, "page_tokens": page_tokens,
            "live": live, "planes": planes, "page_bytes": page_bytes}


def listed():
    return [
        # one user's next token, the usual chat settings: latency alone
        _sample("sample_one_row", 1, 32000, "bf16", "chat"),
        # a few rows whose requests set everything differently, an odd vocabulary, rows at odd offsets,
        # a grammar's mask on some rows and one row it leaves empty
        _sample("sample_mixed_odd", 7, 50257, "f32", "mixed", "grammar"),
        # a server's decode batch under nucleus sampling
        _sample("sample_batch", 64, 131072, "bf16", "nucleus"),
        # the largest decode batch and vocabulary, mixed settings, more than L2 holds
        _sample("sample_large", 256, 262144, "f32", "mixed"),
        # two pages of a small cache: latency alone
        _copy("copy_small", 64, 2, 16, 8192),
        # a prefix of many pages duplicated through every layer's keys and values
        _copy("copy_large", 1024, 509, 64, 32768),
        # four requests, four beams each: the children share full pages and copy the last one
        _fork("fork_beams", 16, 64, 1024, 16, 12, 16, 16384),
        # a large server's step: hundreds of rows forked off long prefixes and every row growing
        _fork("fork_large", 2048, 509, 262147, 16, 512, 2, 2048),
        # a few finished rows of a small server
        _free("free_small", 16, 64, 1024, 16),
        # half of a large server's rows dropped at once
        _free("free_large", 8192, 500, 1048583, 16),
        # a small cache packed
        _compact("compact_small", 16, 64, 1024, 16, 0.5, 4, 4096),
        # a large half-empty cache packed before its upper part is given back
        _compact("compact_large", 1024, 128, 65537, 16, 0.5, 2, 16384),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "copy", "fork", "free", "compact"])
    if op == "sample":
        dtype = rng.choice(["bf16", "f16", "f32"])
        vocab = _log(rng, 1000, 262144)
        rows = _log(rng, 1, max(1, min(256, (64 << 20) // vocab)))
        return _sample("", rows, vocab, dtype, rng.choice(["chat", "mixed", "nucleus", "plain", "greedy"]),
                       rng.choice(["none", "none", "grammar"]))
    if op == "copy":
        planes, page_bytes = _log(rng, 1, 64), rng.choice([48, 1000, 2048, 4100, 8192, 16384, 32768])
        n = _log(rng, 1, max(1, min(500, (1 << 30) // (planes * page_bytes))))
        return _copy("", 2 * n + rng.randrange(1, 30), n, planes, page_bytes)
    page_tokens = rng.choice([1, 8, 16, 16, 32, 64])
    if op == "free":
        rows, width = _log(rng, 1, 8192), _log(rng, 1, 500)
        return _free("", rows, width, rows * width // 2 + 1 + rng.randrange(100), page_tokens)
    if op == "fork":
        rows, width = _log(rng, 2, 2048), _log(rng, 2, 500)
        return _fork("", rows, width, max(8, rows * width // 5 + rng.randrange(100)), page_tokens,
                     rng.randrange(0, rows // 2 + 1), rng.choice([1, 2, 3]), rng.choice([16, 510, 1024, 2048]),
                     rng.choice([0.8, 0.8, 0.98]))
    rows, width = _log(rng, 2, 1024), _log(rng, 2, 128)
    return _compact("", rows, width, max(8, rows * width // 2 + rng.randrange(100)), page_tokens,
                    rng.choice([0.1, 0.5, 0.9]), rng.choice([1, 2]), rng.choice([100, 2048, 16384]))


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


def _prepare_sample(c, g):
    rows, vocab = c["rows"], c["vocab"]
    # a model's logits: a broad bulk, some twenty plausible tokens, in some rows far ahead of the rest
    x = torch.randn(rows, vocab, generator=g, device=DEV).mul_(2.0)
    hot = torch.randint(vocab, (rows, 20), generator=g, device=DEV)
    lift = _uniform(g, rows * 20).view(rows, 20) * 8.0 + _pick(g, rows, [2.0, 5.0, 8.0], torch.float32)[:, None]
    x.scatter_add_(1, hot, lift)
    if c["mask"] == "grammar":
        keep = _uniform(g, rows)[:, None].pow(3)  # the share of the vocabulary a row's grammar allows
        x.masked_fill_(torch.rand(rows, vocab, generator=g, device=DEV) > keep, float("-inf"))
        if rows > 2:
            x[rows // 2] = float("-inf")
    st = {"logits": x.to(DTYPES[c["dtype"]])}
    del x
    # uniform u32 words, held as int32
    st["random"] = torch.randint(-2**31, 2**31, (rows,), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    f32, i32 = torch.float32, torch.int32
    t = {"chat": [0.7, 0.8, 1.0], "mixed": [0.0, 0.5, 0.8, 1.0, 1.5], "nucleus": [0.8, 1.0, 1.2],
         "plain": [0.7, 1.0, 1.3], "greedy": [0.0]}[c["mode"]]
    k = {"chat": [40, 50], "mixed": [0, 0, 1, 20, 50, 1000]}.get(c["mode"])
    p = {"chat": [0.9, 0.95], "mixed": [1.0, 0.5, 0.9, 0.99], "nucleus": [0.8, 0.9, 0.95]}.get(c["mode"])
    a = {"mixed": [0.0, 0.0, 0.02, 0.1]}.get(c["mode"])
    st["temperature"] = _pick(g, rows, t, f32)
    st["top_k"] = _pick(g, rows, k, i32) if k else None
    st["top_p"] = _pick(g, rows, p, f32) if p else None
    st["min_p"] = _pick(g, rows, a, f32) if a else None
    return st


def _pool(g, c):
    """One tensor a plane (a layer's keys or values), as a server holds them."""
    return [torch.randint(-128, 128, (c["pages"], c["page_bytes"]), generator=g, device=DEV, dtype=torch.int8)
            for _ in range(c["planes"])]


def _cache(g, rows, width, pages, page_tokens, budget, live_rows=None):
    """Rows of random lengths over randomly placed pages, at most `budget` of
    them; each odd row shares the first half of the row before it. One int32
    buffer holds table, lens and refs."""
    cap = max(1, min(width, 2 * max(1, budget // max(1, rows)) - 1))
    lens = (_uniform(g, rows) * (cap * page_tokens)).to(torch.int64)
    if live_rows is not None:
        lens[live_rows:] = 0
    n = (lens + page_tokens - 1) // page_tokens
    over = torch.cumsum(n, 0) > budget
    lens[over] = 0
    n[over] = 0
    place = torch.randperm(pages, generator=g, device=DEV)
    mask = torch.arange(width, device=DEV)[None, :] < n[:, None]
    table = torch.full((rows, width), -1, dtype=torch.int64, device=DEV)
    table[mask] = place[: int(n.sum())]
    if rows > 1:
        h = rows // 2
        half = torch.minimum(lens[0 : 2 * h : 2], lens[1 : 2 * h : 2]) // page_tokens // 2
        share = torch.arange(width, device=DEV)[None, :] < half[:, None]
        table[1 : 2 * h : 2] = torch.where(share, table[0 : 2 * h : 2], table[1 : 2 * h : 2])
    refs = torch.bincount(table[table >= 0], minlength=pages)
    return torch.cat([table.flatten(), lens, refs]).to(torch.int32)


def _views(buf, rows, width, pages):
    t = rows * width
    return buf[:t].view(rows, width), buf[t : t + rows], buf[t + rows : t + rows + pages]


def _prepare_cache(c, g):
    rows, width, pages, pt = c["rows"], c["width"], c["pages"], c["page_tokens"]
    st = {"page_tokens": pt}
    if c["op"] == "fork":
        active = rows - c["kids"]
        start = _cache(g, rows, width, pages, pt, int(pages * c["used"]), active)
        _, lens, _ = _views(start, rows, width, pages)
        parent = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
        parent[active:] = torch.randint(active, (rows - active,), generator=g, device=DEV, dtype=torch.int32)
        st["parent"] = parent
        # most rows take one token, some a few (accepted drafts), some a chunk of a prompt, as the row has room
        grow = _pick(g, rows, [1, 1, 1, 1, 4, 5 * pt + 3], torch.int64)
        base = torch.where(parent >= 0, lens[parent.clamp(min=0).long()], lens).long()
        st["grow"] = torch.minimum(grow, width * pt - base).to(torch.int32)
        st["status"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    elif c["op"] == "free":
        start = _cache(g, rows, width, pages, pt, pages - 1)
        st["release"] = (_uniform(g, rows) < 0.5).to(torch.int32)
    else:
        start = _cache(g, rows, width, pages, pt, int(pages * c["live"]))
        st["remap"] = torch.empty(pages, dtype=torch.int32, device=DEV)
    st["start"], st["buf"] = start, start.clone()
    st["table"], st["lens"], st["refs"] = _views(st["buf"], rows, width, pages)
    st["count"] = torch.empty(1, dtype=torch.int32, device=DEV)
    return st


def prepare(case, seed):
    g = _gen(seed)
    c = case
    if c["op"] == "sample":
        st = _prepare_sample(c, g)
        st["tokens"] = torch.empty(c["rows"], dtype=torch.int32, device=DEV)
        st["probs"] = torch.empty(c["rows"], dtype=torch.float32, device=DEV)
    elif c["op"] == "copy":
        perm = torch.randperm(c["pages"], generator=g, device=DEV).to(torch.int32)
        st = {"src": perm[: c["n"]].contiguous(), "dst": perm[c["n"] : 2 * c["n"]].contiguous()}
    else:
        st = _prepare_cache(c, g)
    if "planes" in c:
        st["planes"] = _pool(g, c)
        if own:
            import u32_prefix_scan_gb300 as u

            st["pool"] = u.PagePool(st["planes"])
    st["op"] = c["op"]
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    st = state
    if st["op"] not in ("sample", "copy"):
        st["buf"].copy_(st["start"])  # both forms work in place, each pass from the same cache
    return _RUN_OWN[st["op"]](st) if own else _RUN_PLAIN[st["op"]](st)


def _own_sample(st):
    import u32_prefix_scan_gb300 as u

    return list(u.sample_tokens(st["logits"], st["random"], temperature=st["temperature"], top_k=st["top_k"],
                                top_p=st["top_p"], min_p=st["min_p"], tokens=st["tokens"], probs=st["probs"]))


def _own_copy(st):
    import u32_prefix_scan_gb300 as u

    u.pages_copy(st["pool"], st["src"], st["dst"])
    return st["planes"]


def _own_fork(st):
    import u32_prefix_scan_gb300 as u

    u.pages_fork(st["table"], st["lens"], st["refs"], st["page_tokens"], parent=st["parent"], grow=st["grow"],
                 pool=st["pool"], status=st["status"], free_pages=st["count"])
    return [st["table"], st["lens"], st["refs"], st["status"], st["count"], st["planes"]]


def _own_free(st):
    import u32_prefix_scan_gb300 as u

    u.pages_free(st["table"], st["lens"], st["refs"], st["page_tokens"], st["release"], freed=st["count"])
    return [st["table"], st["lens"], st["refs"], st["count"]]


def _own_compact(st):
    import u32_prefix_scan_gb300 as u

    u.pages_compact(st["pool"], st["table"], st["lens"], st["refs"], st["page_tokens"], live=st["count"],
                    remap=st["remap"])
    return [st["table"], st["lens"], st["refs"], st["count"], st["remap"], st["planes"]]


def _weights(x, m, t):
    """q = floor(2^31 * 2^-y), y = (m - l) log2(e) / T, in single f32 operations."""
    scale = torch.full_like(t, LOG2E) / t
    y = torch.where(x == m, torch.zeros_like(x), (m - x) * scale)
    ok = (y < 32.0) & (x > float("-inf"))
    y = torch.where(ok, y, torch.zeros_like(y))
    n = torch.round(y)
    f = y - n
    p = torch.full_like(f, POLY[4])
    for c in (POLY[3], POLY[2], POLY[1], POLY[0], 1.0):
        p = p * f
        p = p + c
    q = ((p * 2.0**24).to(torch.int64) << 7) >> n.to(torch.int64)
    return torch.where(ok, q, torch.zeros_like(q))


def _plain_sample(st):
    x = st["logits"].float()
    rows, vocab = x.shape
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x)
    m = x.amax(1, keepdim=True)
    index = torch.arange(vocab, device=x.device)
    best = torch.where(x == m, index, vocab).amin(1)
    t = st["temperature"]
    warm = t > 0
    q = _weights(x, m, torch.where(warm, t, torch.ones_like(t))[:, None])
    if st["min_p"] is not None:
        a = st["min_p"].clamp(max=1.0)
        floor = torch.where(a > 0, torch.ceil(a.double() * 2.0**31).to(torch.int64), torch.zeros_like(q[:, 0]))
        q = torch.where(q >= floor[:, None], q, torch.zeros_like(q))
    if st["top_k"] is not None or st["top_p"] is not None:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        qs = q.gather(1, order)
        if st["top_k"] is not None:
            k = torch.where(st["top_k"] > 0, st["top_k"].long(), vocab)
            qs = torch.where(index < k[:, None], qs, torch.zeros_like(qs))
        if st["top_p"] is not None:
            p = st["top_p"].double()
            total = qs.sum(1)
            want = torch.where((p > 0) & (p < 1), torch.ceil(p * total.double()).to(torch.int64), total)
            before = torch.cumsum(qs, 1) - qs
            qs = torch.where(before < want[:, None], qs, torch.zeros_like(qs))
        q = torch.zeros_like(q).scatter_(1, order, qs)
    run_sum = torch.cumsum(q, 1)
    total = run_sum[:, -1]
    word = st["random"].long() & 0xFFFFFFFF
    hi, lo = total >> 25, total & ((1 << 25) - 1)
    r = (word * hi + ((word * lo) >> 25)) >> 7  # floor(word * total / 2^32)
    token = (run_sum <= r[:, None]).sum(1)
    some = m[:, 0] > float("-inf")
    chosen = q.gather(1, token.clamp(max=vocab - 1)[:, None])[:, 0]
    prob = torch.where(warm, chosen.double() / total.clamp(min=1).double(), 1.0)
    st["tokens"].copy_(torch.where(some, torch.where(warm, token, best), -1))
    st["probs"].copy_(torch.where(some, prob, 0.0))
    return [st["tokens"], st["probs"]]


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    for plane in st["planes"]:
        plane[dst] = plane[src]
    return st["planes"]


def _plain_fork(st):
    table, lens, refs = st["table"].long(), st["lens"].long(), st["refs"].long()
    rows, width = table.shape
    pages, pt = refs.numel(), st["page_tokens"]
    parent, grow = st["parent"].long(), st["grow"].long()
    kid = parent >= 0
    par = parent.clamp(0, rows - 1)
    bad = kid & ((parent >= rows) | (lens != 0) | kid[par])
    old = torch.where(kid, lens[par], lens)
    new = old + grow
    held = torch.where(kid, old // pt, (old + pt - 1) // pt)
    bad = bad | (grow < 0) | (old < 0) | ((new + pt - 1) // pt > width)
    need = torch.where(bad, torch.zeros_like(held), (new + pt - 1) // pt - held)
    ends = torch.cumsum(need, 0)
    free = (refs == 0).nonzero()[:, 0]
    served = ~bad & ((need == 0) | (ends <= free.numel()))
    slot = torch.arange(width, device=table.device)[None, :]
    fresh = served[:, None] & (slot >= held[:, None]) & (slot < (held + need)[:, None])
    shared = (served & kid)[:, None] & (slot < held[:, None])
    table = torch.where(shared, table[par], table)
    fresh_pages = free[: int((need * served).sum())]
    table[fresh] = fresh_pages
    entry = table[shared | fresh]
    refs = refs + torch.bincount(entry[(entry >= 0) & (entry < pages)], minlength=pages)
    lens = torch.where(served, new, lens)
    part = (served & kid & (old % pt != 0) & (need > 0)).nonzero()[:, 0]
    src, dst = table[par[part], held[part]], table[part, held[part]]
    for plane in st["planes"]:
        plane[dst] = plane[src]
    status = torch.where(bad, -1, torch.where(served, need, -2))
    st["table"].copy_(table), st["lens"].copy_(lens), st["refs"].copy_(refs)
    st["status"].copy_(status), st["count"].fill_(free.numel() - fresh_pages.numel())
    return [st["table"], st["lens"], st["refs"], st["status"], st["count"], st["planes"]]


def _plain_free(st):
    table, lens, refs = st["table"], st["lens"].long(), st["refs"].long()
    pages, pt = refs.numel(), st["page_tokens"]
    gone = st["release"] != 0
    n = torch.where(gone, (lens + pt - 1) // pt, torch.zeros_like(lens))
    mask = torch.arange(table.shape[1], device=table.device)[None, :] < n[:, None]
    left = refs - torch.bincount(table[mask].long(), minlength=pages)
    st["count"].copy_(((refs > 0) & (left == 0)).sum())
    st["refs"].copy_(left)
    table.masked_fill_(mask, -1)
    st["lens"].masked_fill_(gone, 0)
    return [st["table"], st["lens"], st["refs"], st["count"]]


def _plain_compact(st):
    table, refs = st["table"], st["refs"]
    pages, pt = refs.numel(), st["page_tokens"]
    live = refs != 0
    count = int(live.sum())
    holes = (~live[:count]).nonzero()[:, 0]
    movers = live[count:].nonzero()[:, 0] + count
    remap = torch.where(live, torch.arange(pages, device=refs.device), -1)
    remap[movers] = holes
    for plane in st["planes"]:
        plane[holes] = plane[movers]
    moved = refs[movers]
    refs[movers] = 0
    refs[holes] = moved
    n = (st["lens"].long() + pt - 1) // pt
    mask = torch.arange(table.shape[1], device=table.device)[None, :] < n[:, None]
    table[mask] = remap[table[mask].long()].to(torch.int32)
    st["count"].fill_(count)
    st["remap"].copy_(remap)
    return [st["table"], st["lens"], st["refs"], st["count"], st["remap"], st["planes"]]


_RUN_OWN = {"sample": _own_sample, "copy": _own_copy, "fork": _own_fork, "free": _own_free, "compact": _own_compact}
_RUN_PLAIN = {"sample": _plain_sample, "copy": _plain_copy, "fork": _plain_fork, "free": _plain_free,
              "compact": _plain_compact}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "sample":
        cells = c["rows"] * c["vocab"]
        # a difference, a scaling, the weight's five multiply-adds, its share of the sum
        flops = 0 if c["mode"] == "greedy" else 14 * cells
        return {"bytes": cells * SIZES[c["dtype"]] + 28 * c["rows"], "flops": flops}
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * c["planes"] * c["page_bytes"] + 8 * c["n"], "flops": 0}
    rows, width, pages, pt = c["rows"], c["width"], c["pages"], c["page_tokens"]
    if c["op"] == "fork":
        # refs once, the rows' arguments and results, half a parent's entries a child (read, written, its
        # count raised), the last page of most parents copied
        mean = min(width, 2 * max(1, int(pages * c["used"]) // rows)) / 2
        data = 2 * c["kids"] * (pt - 1) / pt * c["planes"] * c["page_bytes"]
        return {"bytes": int(4 * pages + 24 * rows + c["kids"] * mean * 16 + data), "flops": 0}
    if c["op"] == "free":
        # the released half's entries: read, cleared, their counts lowered
        mean = min(width, 2 * max(1, (pages - 1) // rows)) / 2
        return {"bytes": int(12 * rows + 0.5 * rows * mean * 16), "flops": 0}
    used = min(pages * c["live"], rows * min(width, 2 * max(1, int(pages * c["live"]) // rows)) / 2)
    live = 0.9 * used  # a tenth or so is shared between two rows
    moved = live * (1 - live / pages)
    return {"bytes": int(8 * pages + 4 * rows + 8 * used + moved * (8 + 2 * c["planes"] * c["page_bytes"])), "flops": 0}


# --------------------------------------------------------------------------
# the definitions, one element after another, on the host
# --------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "sample":
        return _exact_sample(c, seed) if c["rows"] * c["vocab"] <= (9 << 20) else None
    if c["op"] == "copy" or c["rows"] * c["width"] > (1 << 18) or c["pages"] > (1 << 18):
        return None
    return {"fork": _exact_fork, "free": _exact_free, "compact": _exact_compact}[c["op"]](c, seed)


def _exact_sample(c, seed):
    st = _prepare_sample(c, _gen(seed))
    logits = st["logits"].float().cpu().numpy()
    words = st["random"].cpu().numpy().view(np.uint32)
    host = {k: None if st[k] is None else st[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p")}
    f32 = np.float32
    out, probs = [], []
    for b in range(c["rows"]):
        x = logits[b]
        x = np.where(np.isnan(x), f32("-inf"), x)
        m = x.max()
        if m == f32("-inf"):
            out.append(-1)
            probs.append(0.0)
            continue
        t = host["temperature"][b]
        if not t > 0:
            out.append(int(np.flatnonzero(x == m)[0]))
            probs.append(1.0)
            continue
        with np.errstate(all="ignore"):
            y = (m - x) * (f32(LOG2E) / t)
        y[x == m] = 0
        near = np.flatnonzero((y < 32) & (x > f32("-inf")))
        y = y[near]
        n = np.rint(y)
        f = y - n
        p = np.full_like(f, f32(POLY[4]))
        for k in (POLY[3], POLY[2], POLY[1], POLY[0], 1.0):
            p = p * f
            p = p + f32(k)
        q = np.floor(p.astype(np.float64) * np.exp2(31.0 - n.astype(np.float64))).astype(np.int64)
        if host["min_p"] is not None and host["min_p"][b] > 0:
            q[q < int(np.ceil(float(min(host["min_p"][b], f32(1))) * 2.0**31))] = 0
        order = np.argsort(-x[near], kind="stable")
        if host["top_k"] is not None and host["top_k"][b] > 0:
            q[order[host["top_k"][b] :]] = 0
        if host["top_p"] is not None and 0 < host["top_p"][b] < 1:
            total = int(q.sum())
            want = int(np.ceil(np.float64(host["top_p"][b]) * np.float64(total)))
            sums = np.cumsum(q[order])
            q[order[int(np.searchsorted(sums, want, side="left")) + 1 :]] = 0
        sums = np.cumsum(q)
        r = (int(words[b]) * int(sums[-1])) >> 32
        at = int(np.searchsorted(sums, r, side="right"))
        out.append(int(near[at]))
        probs.append(int(q[at]) / int(sums[-1]))
    return [torch.tensor(out, dtype=torch.int32), torch.tensor(probs, dtype=torch.float32)]


def _host_cache(c, seed):
    st = _prepare_cache(c, _gen(seed))
    host = {k: v.cpu().numpy().astype(np.int64) for k, v in st.items() if isinstance(v, torch.Tensor)}
    return host, host["table"], host["lens"], host["refs"]


def _i32(*arrays):
    return [torch.from_numpy(np.asarray(a).astype(np.int32).copy()) for a in arrays]


def _exact_fork(c, seed):
    h, table, lens, refs = _host_cache(c, seed)
    pt, width = c["page_tokens"], c["width"]
    parent, grow, before = h["parent"], h["grow"], lens.copy()
    free = [int(i) for i in np.flatnonzero(refs == 0)]
    status, asked, taken = np.zeros(c["rows"], np.int64), 0, 0
    plan = []
    for s in range(c["rows"]):
        p = int(parent[s])
        if p >= 0 and (p >= c["rows"] or before[s] != 0 or parent[p] >= 0):
            status[s] = -1
            continue
        old = int(before[p if p >= 0 else s])
        held = old // pt if p >= 0 else -(-old // pt)
        total = -(-(old + int(grow[s])) // pt)
        if grow[s] < 0 or old < 0 or total > width:
            status[s] = -1
            continue
        need = total - held
        asked += need
        if need > 0 and asked > len(free):
            status[s] = -2
            continue
        status[s] = need
        plan.append((s, p, held, free[asked - need : asked], old + int(grow[s])))
        taken += need
    for s, p, held, fresh, total in plan:
        if p >= 0:
            table[s, :held] = table[p, :held]
            np.add.at(refs, table[p, :held], 1)
        table[s, held : held + len(fresh)] = fresh
        refs[fresh] += 1
        lens[s] = total
    return [*_i32(table, lens, refs, status, [len(free) - taken]), [None] * c["planes"]]


def _exact_free(c, seed):
    h, table, lens, refs = _host_cache(c, seed)
    freed = 0
    for s in np.flatnonzero(h["release"]):
        n = -(-int(lens[s]) // c["page_tokens"])
        for e in table[s, :n]:
            refs[e] -= 1
            freed += int(refs[e] == 0)
        table[s, :n] = -1
        lens[s] = 0
    return _i32(table, lens, refs, [freed])


def _exact_compact(c, seed):
    _, table, lens, refs = _host_cache(c, seed)
    live = int((refs != 0).sum())
    remap = np.where(refs != 0, np.arange(c["pages"]), -1)
    hole = 0
    for p in range(live, c["pages"]):
        if refs[p] != 0:
            while refs[hole] != 0:
                hole += 1
            refs[hole], refs[p], remap[p] = refs[p], 0, hole
    for s in range(c["rows"]):
        n = -(-int(lens[s]) // c["page_tokens"])
        table[s, :n] = remap[table[s, :n]]
    return [*_i32(table, lens, refs, [live], remap), [None] * c["planes"]]
