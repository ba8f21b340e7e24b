"""The step between two decoder calls of a language-model server, on a GPU.

A toy server decodes a few prompts over a paged cache: every step it chooses
each row's next token from its logits (sample_tokens), gives rows the pages
their tokens need and forks some of them into beams (pages_fork), drops the
rows that end (pages_free) and, at the end, packs the cache (pages_compact).
The "model" is a hash of the row's tokens, read back from the cache's pages,
so that a page that went astray would change the text.

    python examples/decode_step.py
"""

import pathlib
import sys

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))

import torch

import u32_prefix_scan_gb300 as u

ROWS, WIDTH, PAGES, PAGE_TOKENS, VOCAB, END, STEPS = 16, 16, 96, 4, 5003, 7, 24


def read_rows(cache, table, lens):
    """The tokens a row's pages hold, -1 past its length: [ROWS, WIDTH * PAGE_TOKENS]."""
    held = cache[table.clamp(min=0).long()].reshape(ROWS, -1)
    at = torch.arange(held.shape[1], device=held.device)
    return torch.where(at < lens[:, None], held, -1)


def toy_logits(tokens):
    """A model's stand-in: peaked logits that depend on every token of the row."""
    h = torch.zeros(tokens.shape[0], dtype=torch.int64, device=tokens.device)
    for column in tokens.unbind(1):
        h = torch.where(column >= 0, (h * 1000003 + column + 1) % 2147483647, h)
    ids = torch.arange(VOCAB, device=tokens.device)
    mixed = (h[:, None] * 48271 + ids * 69621 + 12345) % 2147483647
    return (mixed.double() / 2147483647.0).pow(16).mul(12.0).to(torch.bfloat16)


def main():
    dev = torch.device("cuda")
    cache = torch.full((PAGES, PAGE_TOKENS), -1, dtype=torch.int64, device=dev)  # one plane; a token's own number
    pool = u.PagePool(cache)
    table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(ROWS, dtype=torch.int32, device=dev)
    refs = torch.zeros(PAGES, dtype=torch.int32, device=dev)
    live = torch.zeros(ROWS, dtype=torch.bool, device=dev)
    live[:4] = True
    shadow = [[100 + s] if s < 4 else [] for s in range(ROWS)]  # the same texts, kept by the host

    def write(rows, tokens):
        """Writes each row's newest token into its last page."""
        at = (lens[rows] - 1).long()
        cache[table[rows, at // PAGE_TOKENS].long(), at % PAGE_TOKENS] = tokens.long()

    # the prompts: one token each
    u.pages_fork(table, lens, refs, PAGE_TOKENS, grow=live.int(), pool=pool)
    write(torch.arange(4, device=dev), torch.arange(100, 104, device=dev))

    temperature = torch.full((ROWS,), 0.8, device=dev)
    top_k = torch.full((ROWS,), 40, dtype=torch.int32, device=dev)
    top_p = torch.full((ROWS,), 0.95, device=dev)
    for step in range(STEPS):
        if step == 5:  # the prompts become beams of three
            parent = torch.full((ROWS,), -1, dtype=torch.int32, device=dev)
            parent[4:12] = torch.arange(8, dtype=torch.int32, device=dev) % 4
            parent = torch.where(live[parent.clamp(min=0).long()] & (parent >= 0), parent, -1)
            status, _ = u.pages_fork(table, lens, refs, PAGE_TOKENS, parent=parent, pool=pool)
            live |= (parent >= 0) & (status >= 0)
            for s, p in enumerate(parent.tolist()):
                if p >= 0 and live[s]:
                    shadow[s] = list(shadow[p])
        words = u.fill_splitmix_u32(ROWS, seed=11, stream_id=1, start=step * ROWS, device=dev)
        tokens, _ = u.sample_tokens(toy_logits(read_rows(cache, table, lens)), words, temperature=temperature,
                                    top_k=top_k, top_p=top_p)
        status, free_pages = u.pages_fork(table, lens, refs, PAGE_TOKENS, grow=live.int(), pool=pool)
        live &= status >= 0  # out of pages or out of room: the row ends
        rows = live.nonzero()[:, 0]
        write(rows, tokens[rows])
        for s in rows.tolist():
            shadow[s].append(int(tokens[s]))
        done = live & ((tokens == END) | (tokens % 31 == 0))
        u.pages_free(table, lens, refs, PAGE_TOKENS, done.int())
        live &= ~done
        for s in done.nonzero()[:, 0].tolist():
            shadow[s] = []
    count, _ = u.pages_compact(pool, table, lens, refs, PAGE_TOKENS)
    texts = read_rows(cache, table, lens).tolist()
    for s in live.nonzero()[:, 0].tolist():
        text = [t for t in texts[s] if t >= 0]
        assert text == shadow[s], f"row {s}: {text} is not {shadow[s]}"
        print(f"row {s}: {len(text)} tokens, {' '.join(map(str, text[:8]))} ..")
    assert int(refs[: int(count)].min() if int(count) else 1) > 0 and int(refs[int(count) :].abs().sum()) == 0
    print(f"{int(live.sum())} rows live on {int(count)} of {PAGES} pages")


if __name__ == "__main__":
    main()
