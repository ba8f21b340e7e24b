"""The operators of a decode step together, as a program uses them: rows
forked and grown (pages_fork), keys and values appended to the 8-bit pages
that they got (pages_append), attention over them (pages_attend), rules on the
logits (adjust_logits), the next tokens (sample_tokens), rows released and the
cache packed. Keys, values and scales lie in one page of bytes, so the pool's
operations move them together. Every step is checked against the oracle."""

import numpy as np
import pytest

import oracle
from u32_prefix_scan_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROWS, WIDTH, PAGES, VOCAB = 10, 6, 24, 777
HEADS, GROUP, DIM, PAGE_TOKENS, BLOCKS = 2, 2, 32, 16, 2


@pytest.fixture(scope="module")
def u():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from u32_prefix_scan_gb300 import build

    build.build()
    import u32_prefix_scan_gb300 as u

    return u


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    """A pool whose page holds keys, values and their scales, and the views of it."""

    def __init__(self, u):
        size, scales = PAGE_TOKENS * HEADS * DIM, 4 * BLOCKS * HEADS
        self.bytes = torch.zeros(PAGES, 2 * size + 2 * scales, dtype=torch.uint8, device="cuda")

        def part(at, n, dtype, *shape):
            return self.bytes[:, at : at + n].view(dtype).view(PAGES, *shape)

        e4m3 = torch.float8_e4m3fn
        self.views = [part(0, size, e4m3, PAGE_TOKENS, HEADS, DIM), part(size, size, e4m3, PAGE_TOKENS, HEADS, DIM),
                      part(2 * size, scales, torch.float32, BLOCKS, HEADS),
                      part(2 * size + scales, scales, torch.float32, BLOCKS, HEADS)]
        self.cache = u.KVCache(*self.views)
        self.pool = u.PagePool(self.bytes)

    def host(self):
        k, v, ks, vs = self.views
        return (k.view(torch.uint8).cpu().numpy(), v.view(torch.uint8).cpu().numpy(), ks.cpu().numpy(), vs.cpu().numpy())


def test_steps_of_a_small_server(u):
    rng = np.random.default_rng(1)
    layer = Layer(u)
    table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    angle = np.arange(PAGE_TOKENS * WIDTH)[:, None] * 100.0 ** (-np.arange(DIM // 2) / (DIM // 2))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    cos_d, sin_d = cuda(cos), cuda(sin)
    out_w = torch.from_numpy(rng.standard_normal((HEADS * GROUP * DIM, VOCAB)).astype(np.float32)).cuda()
    history = torch.full((ROWS, PAGE_TOKENS * WIDTH), -1, dtype=torch.int32, device="cuda")
    rules = {"repetition": np.full(ROWS, 1.3, np.float32), "presence": np.full(ROWS, 0.4, np.float32)}
    rules["allowed"] = rng.integers(0, 1 << 32, (ROWS, (VOCAB + 31) // 32), dtype=np.uint64).astype(np.uint32)
    live = np.zeros(ROWS, bool)
    live[:3] = True
    refused = 0
    for step in range(9):
        # prompts first, then a token a row; some steps draft more; one forks, and one asks for more pages than there are
        grow = np.where(live, {0: 21, 4: 3, 7: 40}.get(step, 1), 0).astype(np.int32)
        parent = np.full(ROWS, -1, np.int32)
        if step == 3:
            parent[3:9] = [0, 1, 2, 0, 1, 2]
            live[3:9] = True
            grow[3:9] = 1
        kw = {} if step != 3 else {"parent": cuda(parent)}
        status, _ = u.pages_fork(table, lens, refs, PAGE_TOKENS, grow=cuda(grow), pool=layer.pool, **kw)
        starts = np.concatenate([[0], np.cumsum(grow)]).astype(np.int32)
        tokens = int(starts[-1])
        qkv = torch.from_numpy(rng.standard_normal((tokens, HEADS * (GROUP + 2), DIM)).astype(np.float32)).bfloat16()
        q, k, v = qkv.cuda().split([HEADS * GROUP, HEADS, HEADS], 1)
        before = layer.host()
        turned = u.pages_append(layer.cache, table, lens, k, v, starts=cuda(starts), status=status, cos=cos_d, sin=sin_d,
                                queries=q)
        out = u.pages_attend(layer.cache, table, lens, turned, starts=cuda(starts))

        # the cache and the queries, bit for bit
        t, n, st = table.cpu().numpy(), lens.cpu().numpy(), status.cpu().numpy()
        refused += int((st < 0).sum())
        served = [s for s in range(ROWS) if grow[s] and st[s] >= 0]
        want = oracle.pages_append(before[0], before[1], t, n, k.float().cpu().numpy(), v.float().cpu().numpy(), starts, st,
                                   cos, sin, False, before[2], before[3], q.float().cpu().numpy(),
                                   np.zeros((tokens, HEADS * GROUP, DIM), np.float32))
        for got, exact in zip(layer.host(), want):
            assert np.array_equal(got, exact)
        rows = np.concatenate([np.arange(starts[s], starts[s + 1]) for s in served])
        assert torch.equal(turned.cpu()[rows], torch.from_numpy(want[4]).bfloat16()[rows])
        live &= st >= 0
        # attention to its arithmetic: weights to 2^-11, scores to f32, the result to half a bf16 step (2^-8)
        exact = oracle.pages_attend(turned.double().cpu().numpy(), *want[:4], t, n, starts)
        mags = oracle.pages_attend(turned.double().cpu().numpy(), want[0], want[1] & 0x7F, *want[2:4], t, n, starts)
        off = np.abs(out.double().cpu().numpy() - exact)
        assert np.all(off[rows] <= mags[rows] * 2.0**-10 + 2.0**-8 * np.abs(exact[rows]) + 1e-6)

        # each row's last token, its rules, and the draw
        last = cuda(np.maximum(starts[1:] - 1, 0).astype(np.int64))
        logits = (out[last].nan_to_num().float().flatten(1) @ out_w).bfloat16()
        lens_h = cuda(np.where(live, n, 0).astype(np.int32))
        words = inputs.splitmix_u32(5, step, ROWS)
        fixed = {k2: cuda(v2.view(np.int32) if v2.dtype == np.uint32 else v2) for k2, v2 in rules.items()}
        ruled = u.adjust_logits(logits, history=history, history_lens=lens_h, out=logits.clone(), **fixed)
        u.adjust_logits(logits, history=history, history_lens=lens_h, out=logits, **fixed)  # in place, the same
        assert torch.equal(ruled, logits)
        drawn, _ = u.sample_tokens(ruled, cuda(words.view(np.int32)))
        want_tokens, _ = oracle.sample_tokens(ruled.float().cpu().numpy(), words)
        assert np.array_equal(drawn.cpu().numpy(), want_tokens)
        allowed = rules["allowed"][np.arange(ROWS), np.maximum(want_tokens, 0) // 32] >> (np.maximum(want_tokens, 0) % 32).astype(np.uint32) & 1
        assert np.all(allowed == 1)
        for s in served:
            history[s, n[s] - grow[s] : n[s]] = int(want_tokens[s])

        if step in (5, 8):  # some rows end; what is left moves to the front and attends to the same
            gone = np.zeros(ROWS, np.int32)
            gone[[1, 4]] = 1
            u.pages_free(table, lens, refs, PAGE_TOKENS, cuda(gone))
            live &= gone == 0
            kept = [s for s in served if live[s]]
            one = cuda(np.arange(ROWS + 1, dtype=np.int32))
            probe = turned[last].nan_to_num()
            first = u.pages_attend(layer.cache, table, lens, probe, starts=one)
            u.pages_compact(layer.pool, table, lens, refs, PAGE_TOKENS)
            again = u.pages_attend(layer.cache, table, lens, probe, starts=one)
            assert torch.equal(first, again) and first[kept].abs().sum() > 0
    assert refused > 0 and live.sum() >= 2  # rows were refused their pages on the way, and left as they were
