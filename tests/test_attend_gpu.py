"""GPU parity of pages_attend against attention in 64 bits: head layouts,
lengths from none to long, pages and blocks of any size in any order, drafts,
masked places that hold NaN, strides."""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def u():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from u32_prefix_scan_gb300 import build

    build.build()
    import u32_prefix_scan_gb300 as u

    return u


class Case:
    def __init__(self, seed, lens, counts=None, *, heads=2, group=2, dim=64, page_tokens=16, blocks=1, dtype="bf16",
                 spare=2, tail=0, peaked=1.0, scales=(-9, -5)):
        rng = np.random.default_rng(seed)
        self.dtype, self.dim = dtype, dim
        self.lens = np.asarray(lens, np.int32)
        rows = len(lens)
        need = -(-np.maximum(self.lens, 0) // page_tokens)
        self.pages = int(need.sum()) + spare
        self.table = np.full((rows, max(int(need.max(initial=0)), 1)), -1, np.int32)
        place, at = rng.permutation(self.pages), 0
        for s in range(rows):
            self.table[s, : need[s]] = place[at : at + need[s]]
            at += need[s]
        self.starts = None if counts is None else np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.tokens = rows if counts is None else int(np.sum(counts)) + tail
        shape = (self.pages, page_tokens, heads, dim)
        x = np.clip(rng.standard_normal((2, *shape)) * 110, -448, 448).astype(np.float32)
        self.keys, self.values = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        s = rng.integers(*scales, (2, self.pages, blocks, heads))
        self.key_scales, self.value_scales = (np.exp2(s) * rng.choice([1.0, 1.0, 0.7], s.shape)).astype(np.float32)
        q = rng.standard_normal((self.tokens, heads * group, dim)) * peaked
        self.queries = torch.from_numpy(q.astype(np.float32)).to(TYPES[dtype])
        self.scale = None
        self.extra = 0.0

    def gpu(self):
        def dev(a):
            return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()

        d = {k: dev(getattr(self, k)) for k in ("table", "lens", "starts", "key_scales", "value_scales")}
        d["keys"], d["values"] = (dev(getattr(self, k)).view(torch.float8_e4m3fn) for k in ("keys", "values"))
        d["queries"] = self.queries.cuda()
        return d

    def arrays(self, values=None, **kw):
        args = dict(scale=self.scale, starts=self.starts) | kw
        return oracle.pages_attend(self.queries.double().numpy(), self.keys, self.values if values is None else values,
                                   self.key_scales, self.value_scales, self.table, self.lens, **args)

    def check(self, got):
        """The result's error, first order: each weight is rounded to f16 (2^-11
        relative), so the sum is off by 2^-11 of the weighted magnitudes;
        weights below f16's normal range (2^-14 of the weight last taken as
        1) are off by 2^-25 each, times a code of at most 448 and its scale;
        a score s is off by its f32 sum of dim products and the few roundings
        after it, (dim + 8) 2^-24 of its sum of magnitudes, and exp2 of
        that by twice as much on both sides of the quotient; last the
        result's own rounding, half a step."""
        want = self.arrays()
        some = np.isfinite(want)
        if not some.any():
            return want
        mags = self.arrays(values=self.values & 0x7F)
        q, pages = np.abs(self.queries.double().numpy()), self.table[self.table >= 0]
        pages = pages[pages < self.pages]
        top = 448.0 * (self.value_scales[pages].max() if pages.size else 0.0)
        dots = q.sum(-1).max() * 448.0 * (self.key_scales[pages].max() if pages.size else 0.0)
        dots *= self.dim**-0.5 if self.scale is None else abs(self.scale)
        # a sum of products of any sign is far from its magnitudes' bound: the dim roundings add like sqrt(dim)
        score = (np.sqrt(self.dim) + 8) * 2.0**-24 * dots / np.sqrt(self.dim) * 4
        longest = max(int(self.lens.max(initial=0)), 1)
        half = float(torch.finfo(TYPES[self.dtype]).eps) / 2
        tol = mags * (2.0**-11 + 2 * score + 2.0**-18) + longest * 2.0**-25 * top + half * np.abs(want) + self.extra
        off = np.abs(got.double().cpu().numpy() - want)
        assert np.isfinite(got.float().cpu().numpy()[some]).all()
        assert np.all(off[some] <= tol[some]), (off[some] / tol[some]).max()
        return want


def call(u, d, **kw):
    cache = u.KVCache(d["keys"], d["values"], d["key_scales"], d["value_scales"])
    out = u.pages_attend(cache, d["table"], d["lens"], d["queries"], **{"starts": d["starts"], **kw})
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 240, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 9, 16, 20])
def test_dims_and_groups(u, dim, group, dtype):
    c = Case(dim + group, [77, 1, 33, 200], dim=dim, group=group, dtype=dtype, heads=3 if group < 8 else 1)
    c.check(call(u, c.gpu()))


@pytest.mark.parametrize("page_tokens,blocks", [(1, 1), (3, 3), (4, 1), (10, 2), (16, 16), (16, 1), (20, 2), (24, 1),
                                               (48, 3), (64, 1), (64, 8), (100, 4), (128, 2)])
@pytest.mark.parametrize("dim", [64, 128])
def test_pages_and_blocks(u, page_tokens, blocks, dim):
    c = Case(page_tokens, [1, 2, 15, 16, 17, 63, 64, 65, 300], page_tokens=page_tokens, blocks=blocks, dim=dim)
    c.check(call(u, c.gpu()))


@pytest.mark.parametrize("length", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 64, 127, 128, 129, 500, 1023, 4097])
def test_one_row_of_every_length(u, length):
    c = Case(length, [length], heads=4, group=4, dim=128)
    c.check(call(u, c.gpu()))


@pytest.mark.parametrize("rows,length", [(1, 40001), (3, 30000), (300, 700)])
def test_long_and_many(u, rows, length):
    lens = np.linspace(1, length, rows).astype(int)[::-1]
    c = Case(rows, lens, heads=1, group=2, dim=64, page_tokens=32)
    c.check(call(u, c.gpu()))


@pytest.mark.parametrize("length,heads,drafts,group,dim", [(60000, 1, 5, 7, 64), (50000, 2, 1, 8, 128), (30000, 4, 3, 5, 128)])
def test_one_long_row_in_many_parts(u, length, heads, drafts, group, dim):
    """A row's tiles of queries cut into more parts than are joined at a time."""
    c = Case(length, [length], [drafts], heads=heads, group=group, dim=dim, page_tokens=16)
    c.check(call(u, c.gpu()))


@pytest.mark.parametrize("rows", [255, 256, 257, 700])
def test_rows_more_than_threads(u, rows):
    lens = np.arange(rows) * 37 % 90
    c = Case(rows, lens, heads=4, group=1, dim=64, page_tokens=8)
    c.check(call(u, c.gpu()))


@pytest.mark.parametrize("counts", [[1, 1, 1], [5, 1, 3], [0, 7, 0], [16, 33, 2], [70, 9, 80]])
@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (7, 64), (8, 256), (2, 96)])
def test_drafts(u, counts, group, dim):
    c = Case(group, [90, 40, 120], counts, group=group, dim=dim, page_tokens=10, blocks=2)
    c.check(call(u, c.gpu()))


def test_rows_and_queries_that_see_nothing(u):
    """Empty rows, rows shorter than their new tokens, rows without pages:
    zeros; tokens behind the last row's are left alone."""
    c = Case(2, [0, 40, 3, 25, 30], [2, 3, 7, 1, 1], tail=4, heads=2, group=3)
    c.table[3] = -1
    c.table[4, 0], c.table[4, 1] = c.pages, -7  # a page's worth missing at both ends
    d = c.gpu()
    out = torch.full_like(d["queries"], 5.0)
    assert call(u, d, out=out) is out
    want = c.check(out)
    got = out.float().cpu().numpy()
    assert np.all(got[-4:] == 5) and np.isnan(want[-4:]).all()
    assert not got[:2].any() and not got[5:9].any() and not got[12].any()  # an empty row; 4 of 7; no pages
    assert not got[13].any()  # its only two pages are not the pool's


def test_pages_missing_in_the_middle(u):
    c = Case(4, [100, 64], page_tokens=8, dim=128)
    c.table[0, 3], c.table[0, 11], c.table[1, 0] = -1, c.pages + 5, -1
    c.check(call(u, c.gpu()))


def test_lens_past_the_table(u):
    c = Case(5, [100, 64], page_tokens=8)
    c.lens[0] = 2**31 - 1
    d = c.gpu()
    got = call(u, d)
    c.lens[0] = 104  # what the table holds
    c.check(got)


@pytest.mark.parametrize("dim,group", [(64, 2), (128, 8), (256, 4)])
def test_nan_in_masked_places(u, dim, group):
    """Slots past a row's length, pages of nobody, and drafts that a query does
    not see yet may hold anything."""
    c = Case(6, [37, 20, 50], [4, 1, 9], dim=dim, group=group)
    d = c.gpu()
    clean = call(u, d)
    for s, (length, n) in enumerate(zip(c.lens, np.diff(c.starts))):
        page, slot = c.table[s, (length - 1) // 16], (length - 1) % 16
        for k in ("keys", "values"):
            t = d[k].view(torch.uint8)
            t[page, slot + 1 :] = 0x7F
            t[page, slot] = 0xFF  # the last token: only the last query sees it
    used = set(c.table[c.table >= 0].tolist())
    for p in set(range(c.pages)) - used:
        d["keys"].view(torch.uint8)[p] = 0x7F
        d["values"].view(torch.uint8)[p] = 0x7F
        d["key_scales"][p] = float("nan")
        d["value_scales"][p] = float("inf")
    got = call(u, d)
    last = c.starts[1:] - 1
    rest = np.setdiff1d(np.arange(c.tokens), last)
    assert torch.equal(got[rest], clean[rest])
    assert got[last].isnan().all()


@pytest.mark.parametrize("which", ["keys", "values"])
def test_nan_that_is_seen(u, which):
    c = Case(7, [50, 20], [6, 1])
    d = c.gpu()
    d[which].view(torch.uint8)[c.table[0, 47 // 16], 47 % 16, 1, 5] = 0x7F  # position 47 of 50, head 1, element 5
    got = call(u, d).float()
    nan = got.isnan().cpu().numpy()
    want = np.zeros_like(nan)
    if which == "keys":
        want[3:6, 2:4] = True
    else:
        want[3:6, 2:4, 5] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("scales", [(-100, -90), (-40, 30), (60, 80)])
@pytest.mark.parametrize("which", ["key_scales", "value_scales"])
def test_scales_far_apart(u, which, scales):
    """Blocks whose scales lie many powers apart: of keys, one token takes all;
    of values, the weights must not lose the small ones' softmax sum."""
    c = Case(8, [200, 33], page_tokens=8, dim=64, blocks=2)
    rng = np.random.default_rng(1)
    s = getattr(c, which)
    s[...] = np.exp2(rng.integers(*scales, s.shape)).astype(np.float32)
    if which == "key_scales":
        c.queries = (c.queries.float() * 2.0 ** -float(scales[1])).to(c.queries.dtype)
        if scales[1] > 40 or scales[0] < -90:
            c.queries = (torch.sign(c.queries.float()) * 2.0 ** -min(scales[1], 14)).to(c.queries.dtype)
            s *= np.float32(2.0 ** (-scales[1] + 4))
    if scales[1] > 20 and which == "value_scales":
        s *= np.float32(2.0 ** -scales[1])
    c.check(call(u, c.gpu()))


def test_blocks_of_zero(u):
    """Zero scales: a key's score is 0, a value's share is nothing but counts."""
    c = Case(9, [64, 20], page_tokens=16)
    c.key_scales[c.table[0, 1]] = 0.0
    c.value_scales[c.table[0, 2]] = 0.0
    c.value_scales[c.table[1]] = 0.0
    got = call(u, c.gpu())
    c.check(got)
    assert not got[1].any()


@pytest.mark.parametrize("peaked", [0.0, 30.0, 2000.0])
def test_flat_and_peaked(u, peaked):
    c = Case(10, [1000, 17], peaked=peaked, dim=128, scales=(-7, -6))
    if peaked > 100:  # a score's rounding decides nothing where one token takes all: leave the ties out
        c.scale = 1e-3
    c.check(call(u, c.gpu(), scale=c.scale))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scale(u, scale):
    c = Case(12, [130, 65])
    c.scale = scale
    c.check(call(u, c.gpu(), scale=scale))


def test_query_magnitudes(u):
    """Heads of queries from 2^-100 to 2^100 (bf16) meet scales that balance them."""
    c = Case(13, [90, 90, 90, 90, 90], heads=1, group=1)
    for s, e in enumerate((-100, -30, 0, 30, 100)):
        c.queries[s] = (c.queries[s].float() * 2.0**e).bfloat16()
        used = c.table[s][c.table[s] >= 0]
        c.key_scales[used] *= np.float32(2.0) ** -e
    got = call(u, c.gpu())
    want = c.arrays()
    mags = c.arrays(values=c.values & 0x7F)
    # the plain scores' errors, as check() states them for the row of e = 0
    off = np.abs(got.double().cpu().numpy() - want) / (mags * (2.0**-11 + 2.0**-12) + 2.0**-8 * np.abs(want))
    assert off.max() <= 1, off.max((1, 2))  # (bf16: half a step is eps / 2 = 2^-8)


@pytest.mark.parametrize("layout", ["heads_first", "one_page", "gaps"])
def test_layouts(u, layout):
    """Heads before tokens; keys, values and scales in one page of bytes; room
    between everything. Queries and outputs with strides of their own."""
    c = Case(14, [70, 45], [3, 2], heads=2, dim=64, page_tokens=16, blocks=2)
    d = c.gpu()
    plain = call(u, d)
    size = 16 * 2 * 64
    if layout == "heads_first":
        for k in ("keys", "values"):
            d[k] = d[k].transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "one_page":
        room = torch.zeros(c.pages, 2 * size + 2 * 16, dtype=torch.uint8, device="cuda")
        for i, k in enumerate(("keys", "values")):
            view = room[:, i * size : (i + 1) * size].view(torch.float8_e4m3fn).view(c.pages, 16, 2, 64)
            view.view(torch.uint8).copy_(d[k].view(torch.uint8))
            d[k] = view
            at = 2 * size + 16 * i
            s = room[:, at : at + 16].view(torch.float32).view(c.pages, 2, 2)
            s.copy_(d[k[:-1] + "_scales"])
            d[k[:-1] + "_scales"] = s
    else:
        for k in ("keys", "values"):
            room = torch.zeros(c.pages, 18, 3, 96, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            view = room[:, 1:17, :2, 16:80]
            view.copy_(d[k])
            d[k] = view
        q = torch.zeros(c.tokens, 6, 72, dtype=torch.bfloat16, device="cuda")[:, 1:5, 8:]
        q.copy_(d["queries"])
        d["queries"] = q
    out = torch.full((c.tokens, 4, 65), 3.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(call(u, d, out=out[:, :, 1:]), plain)
    assert torch.all(out[:, :, 0] == 3)


def test_the_same_twice(u):
    """Bits do not depend on what ran before, nor on the stream."""
    c = Case(15, np.arange(1, 2000, 97), heads=2, group=5, dim=128)
    d = c.gpu()
    first = call(u, d)
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        got = call(u, d, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, first)


def test_graphs_that_share_a_workspace(u):
    """Two captured calls on one stream's workspace, replayed in turn with other lengths and queries."""
    a, b = Case(16, [900, 30, 400], heads=2, group=4, dim=128), Case(17, [50] * 20, heads=1, group=2, dim=64)
    da, db = a.gpu(), b.gpu()
    call(u, da), call(u, db)
    ws = u.Workspace.get(10, 1, torch.device("cuda", 0), torch.cuda.current_stream().cuda_stream)
    graphs, outs = [], []
    for d in (da, db):
        cache = u.KVCache(d["keys"], d["values"], d["key_scales"], d["value_scales"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(u.pages_attend(cache, d["table"], d["lens"], d["queries"], workspace=ws))
        graphs.append((graph, cache))
    for turn in range(2):
        a.lens -= 100 * turn
        a.lens[:] = np.maximum(a.lens, 0)
        a.queries = a.queries * (1 + turn)
        da["lens"].copy_(torch.from_numpy(a.lens))
        da["queries"].copy_(a.queries)
        graphs[0][0].replay()
        graphs[1][0].replay()
        torch.cuda.synchronize()
        a.check(outs[0])
        b.check(outs[1])


def test_none_of_it(u):
    c = Case(18, [30], dim=64)
    d = c.gpu()
    q = d["queries"][:0]
    cache = u.KVCache(d["keys"], d["values"], d["key_scales"], d["value_scales"])
    assert u.pages_attend(cache, d["table"][:0], d["lens"][:0], q).shape == q.shape
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert u.pages_attend(cache, d["table"], d["lens"], q, starts=zero).shape == q.shape
    empty = u.KVCache(d["keys"][:0], d["values"][:0], d["key_scales"][:0], d["value_scales"][:0])
    assert not u.pages_attend(empty, d["table"], d["lens"], d["queries"]).any()
    no_width = u.pages_attend(cache, d["table"][:, :0], d["lens"], d["queries"])
    assert not no_width.any()


def test_a_workspace_shared_with_other_operations(u):
    """Scans, sorts and page operations leave their words and buffers where the
    call keeps its counts and partial sums, and the other way round."""
    from u32_prefix_scan_gb300 import _native, inputs

    c = Case(19, [900, 30, 400, 77], heads=4, group=4, dim=128)
    d = c.gpu()
    want = call(u, d)
    n = (1 << 20) + 77
    sizes = [(1, n), (4, n), (9, 500), (10, 1)]
    ws = u.Workspace(max(_native.lib().u32scan_workspace_bytes(*s) for s in sizes), torch.device("cuda"))
    values = inputs.splitmix_u32(7, 0, n)
    scanned, total = oracle.scan_exclusive(values)
    refs = torch.zeros(400, dtype=torch.int32, device="cuda")
    for _ in range(3):
        a = torch.from_numpy(values.view(np.int32).copy()).cuda()
        u.scan_exclusive_u32(a, workspace=ws)
        assert torch.equal(call(u, d, workspace=ws), want)
        perm = u.radix_sort_perm_u32(torch.from_numpy(values.view(np.int32).copy()).cuda(), workspace=ws)
        assert torch.equal(call(u, d, workspace=ws), want)
        lens, table = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.full((5, 4), -1, dtype=torch.int32, device="cuda")
        status, _ = u.pages_fork(table, lens, refs * 0, 16, grow=lens + 20, workspace=ws)
        assert torch.equal(call(u, d, workspace=ws), want)
        assert np.array_equal(a.cpu().numpy().view(np.uint32), scanned) and status.tolist() == [2] * 5
        assert np.array_equal(perm.cpu().numpy(), oracle.sort_perm(values))
    assert u.check(workspace=ws) == _native.OK


def test_the_end_of_a_tag_period(u):
    """The launch that ends a period of tags clears the counts, so that the
    same tags start from none."""
    c = Case(20, [5000, 3000], heads=2, group=4, dim=128)
    d = c.gpu()
    want = call(u, d)
    ws = u.Workspace(u._native.lib().u32scan_workspace_bytes(10, 1), torch.device("cuda"))

    def set_epoch(e):
        ws.buf[4:8].copy_(torch.tensor([e], dtype=torch.int64).to(torch.int32).view(torch.uint8))

    period = 1 << 29
    for start in (period - 2, 2 * period - 2, 3 * period - 2):
        set_epoch(start)
        for _ in range(4):  # two before the period's end, two behind
            assert torch.equal(call(u, d, workspace=ws), want)
        head = ws.buf[:8].view(torch.int32).tolist()
        assert head[0] == 0 and head[1] & 0xFFFFFFFF == start + 4


@pytest.mark.parametrize("page_tokens", [16, 20])
def test_offsets_past_32_bits(u, page_tokens):
    """Pages half a gigabyte apart."""
    c = Case(23, [page_tokens * 4 + 3, 50], [2, 1], heads=2, group=3, dim=64, page_tokens=page_tokens)
    d = c.gpu()
    room = torch.empty(c.pages << 29, dtype=torch.uint8, device="cuda").view(c.pages, 1 << 29)
    assert room.numel() > 1 << 32
    size = page_tokens * 2 * 64
    for at, k in ((0, "keys"), (1 << 28, "values")):
        view = room[:, at : at + size].view(torch.float8_e4m3fn).view(c.pages, page_tokens, 2, 64)
        view.view(torch.uint8).copy_(d[k].view(torch.uint8))
        d[k] = view
    c.check(call(u, d))


def test_two_streams_at_once(u):
    """Each stream has a workspace of its own; neither call sees the other's."""
    cases = [Case(24, [3000, 20, 700], heads=4, group=4, dim=128), Case(25, [1500] * 9, [3] * 9, heads=2, group=2, dim=64)]
    ds = [c.gpu() for c in cases]
    want = [call(u, d) for d in ds]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for i, (d, s) in enumerate(zip(ds, streams)):
            cache = u.KVCache(d["keys"], d["values"], d["key_scales"], d["value_scales"])
            outs[i].append(u.pages_attend(cache, d["table"], d["lens"], d["queries"], starts=d["starts"], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("page_tokens,blocks", [(16, 2), (16, 16), (48, 2), (32, 4), (20, 2)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 8), (256, 4)])
def test_scales_of_unwritten_blocks(u, page_tokens, blocks, poison, dim, group):
    """A row's last page may hold blocks that no token was written to: their scales are anybody's."""
    c = Case(26, [5, 20, 50, 33], [1, 3, 9, 1], dim=dim, group=group, page_tokens=page_tokens, blocks=blocks)
    d = c.gpu()
    clean = call(u, d)
    c.check(clean)
    size, poisoned = page_tokens // blocks, 0
    for s, length in enumerate(c.lens):
        page, nth = c.table[s, (length - 1) // page_tokens], (length - 1) % page_tokens // size
        for k in ("key_scales", "value_scales"):
            d[k][page, nth + 1 :] = poison
            poisoned += blocks - 1 - nth
    assert poisoned > 0
    assert torch.equal(call(u, d), clean)


@pytest.mark.parametrize("which", ["key_scales", "value_scales"])
def test_scales_of_drafts_not_seen_yet(u, which):
    """A block that holds a row's last draft alone: only that draft meets its scale."""
    c = Case(27, [41, 25], [6, 2], page_tokens=16, blocks=2)
    d = c.gpu()
    clean = call(u, d)
    for s, length in enumerate(c.lens):
        d[which][c.table[s, (length - 1) // 16], (length - 1) % 16 // 8] = float("nan")
    got = call(u, d)
    last = c.starts[1:] - 1
    rest = np.setdiff1d(np.arange(c.tokens), last)
    assert torch.equal(got[rest], clean[rest])
    assert got[last].isnan().all()


def test_a_small_weight_meets_a_large_scale(u):
    """A warp's first tile has values of 0 at the least scale; in its next one the weights are 0 in
    f32 and the scale is large: their product is nothing."""
    rows = 320  # so that a block has whole rows
    c = Case(28, [144] * rows, heads=1, group=1, dim=64)
    c.table[:] = c.table[0]
    c.keys[...] = 0
    c.keys[c.table[0, 0], 0] = 0x38  # token 0's score is 3 * 8 * 64, the others' 0: e^-1536
    c.key_scales[...] = 1.0
    c.queries[...] = 8.0
    c.values[c.table[0, 0]] = 0
    c.value_scales[...] = 1.0
    c.value_scales[c.table[0, 0]] = 2.0**-100
    c.value_scales[c.table[0, 8]] = 2.0**30  # tokens 128 to 143: the same warp's next tile
    assert not call(u, c.gpu(), scale=3.0).any()


def own_bound(c, got):
    """The largest quotient of a result's error, against attention in 64 bits, and its bound. With w_j
    the tokens' softmax weights, v_j their codes, s_j the scales of their values' blocks and H the largest
    w_j s_j of the query: a weight is rounded to f16, to 2^-11 of itself or, below f16's normal
    range, half of f16's least step, 2^-25, where H has become 2^7 at least: 2^-32 H. A score is off by
    its f32 sum of dim products and the roundings after it, (dim + 8) 2^-23 of its sum of magnitudes (a step a sum,
    whichever way they are rounded), which acts on both sides of the quotient. 2^-18 for the sums of products, and half a step (f16: 2^-25 at least)
    of the result's own."""
    worst, got = 0.0, got.double().cpu().numpy()
    page_tokens, heads = c.keys.shape[1:3]
    size = page_tokens // c.key_scales.shape[1]
    tokens, q_heads, dim = c.queries.shape
    group = q_heads // heads
    half = float(torch.finfo(TYPES[c.dtype]).eps) / 2
    codes = oracle.code_values(np.arange(256)).astype(np.float64)
    starts = np.arange(len(c.lens) + 1) if c.starts is None else c.starts
    scale = c.dim**-0.5 if c.scale is None else c.scale
    for row, length in enumerate(c.lens):
        at = np.arange(min(int(length), c.table.shape[1] * page_tokens))
        page = c.table[row, at // page_tokens]
        placed = (page >= 0) & (page < c.pages)
        at, page = at[placed], page[placed]
        slot = at % page_tokens
        for h in range(heads):
            ks, vs = (t[page, slot // size, h].astype(np.float64) for t in (c.key_scales, c.value_scales))
            k, v = codes[c.keys[page, slot, h]] * ks[:, None], codes[c.values[page, slot, h]]
            size_of_v = np.abs(v)
            for token in range(starts[row], starts[row + 1]):
                n = int((at <= length - starts[row + 1] + token).sum())
                q = c.queries[token, h * group : (h + 1) * group].double().numpy()
                its = got[token, h * group : (h + 1) * group]
                if n == 0:
                    assert not its.any()
                    continue
                s = q @ k[:n].T * scale
                score = (dim + 8) * 2.0**-23 * (np.abs(q) @ np.abs(k[:n]).T).max() * abs(scale)
                w = np.exp(s - s.max(1, keepdims=True))
                w = w / w.sum(1, keepdims=True) * vs[:n]
                want = w @ v[:n]
                tol = (w @ size_of_v[:n]) * (2.0**-11 + 2.0**-18 + 2 * score) + half * np.abs(want)
                tol += 2.0**-32 * w.max(1)[:, None] * size_of_v[:n].sum(0) + 2.0**-25
                off = np.abs(its - want)
                assert np.isfinite(off).all()
                worst = max(worst, float((off / tol).max()))
    return worst


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("gap", [12, 18, 24, 26])
@pytest.mark.parametrize("length", [128, 5000])
def test_many_small_weights_beside_sinks(u, length, gap, dtype):
    """One token of every 16 takes all the weight, and its value is 0: what comes out is the others'."""
    c = Case(29, [length], heads=1, group=2, dim=64, dtype=dtype)
    c.keys[...] = 0
    c.keys[:, 0] = 0x38  # 1
    c.key_scales[...] = 1.0
    c.queries[...] = 1.0
    c.scale = gap * float(np.log(2)) / 64  # the others' weight: 2^-gap
    c.values[...] = np.random.default_rng(gap).integers(0x70, 0x7F, c.values.shape)  # 128 to 448
    c.values[:, 0] = 0
    c.value_scales[...] = 2.0 ** min(gap - 9, 7)  # (the results lie in f16's normal range)
    worst = own_bound(c, call(u, c.gpu(), scale=c.scale))
    assert worst <= 1, worst


@pytest.mark.parametrize("low", [20, 99, 110, 127])
def test_scores_far_below_zero(u, low):
    """Equal scores weigh the same, however low they are; a row's only token weighs 1."""
    c = Case(30, [40, 700, 1], heads=2, group=2, dim=64)
    c.keys[...] = 0x38
    c.key_scales[...] = 1.0
    c.queries[...] = -(2.0 ** (low - 6))  # scores of -2^low
    got = call(u, c.gpu(), scale=1.0)
    c.queries[...] = 0.0
    c.scale = 1.0
    worst = own_bound(c, got)
    assert worst <= 1, worst


def segments(c):
    """Values that tell their places: token j of a row has one element that is not 0, the one of its share of the row."""
    page_tokens, heads, dim = c.keys.shape[1:]
    rng = np.random.default_rng(len(c.lens))
    c.values[...] = 0
    for row, length in enumerate(c.lens):
        at = np.arange(int(length))
        page, d = c.table[row, at // page_tokens], at * dim // max(int(length), 1)
        ok = page >= 0
        for h in range(heads):
            c.values[page[ok], at[ok] % page_tokens, h, d[ok]] = rng.integers(0x60, 0x7F, int(ok.sum()))
    return c


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("length,heads,drafts,group,dim", [(60000, 1, 5, 7, 64), (50000, 2, 1, 8, 128), (30000, 4, 3, 5, 128),
                                                          (20000, 2, 2, 3, 256), (40000, 1, 1, 16, 80)])
def test_every_token_of_a_long_row_counts(u, length, heads, drafts, group, dim, dtype):
    """A part that is lost, or joined with a wrong weight, is missed in its tokens' own elements."""
    c = segments(Case(length, [length], [drafts], heads=heads, group=group, dim=dim, dtype=dtype))
    worst = own_bound(c, call(u, c.gpu()))
    assert worst <= 1, worst


# heads beside each other in a block: 4 for 8 x 8 and 4 x 3, 2 for six heads, two heads, 256 dimensions and groups of 16
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,length,heads,group,dim,page_tokens,blocks", [
    (64, 2500, 8, 8, 128, 16, 1), (40, 2000, 4, 3, 64, 32, 2), (40, 1500, 6, 2, 128, 64, 4), (80, 1800, 2, 4, 64, 16, 2),
    (48, 700, 8, 1, 256, 16, 1), (60, 1200, 4, 16, 128, 32, 2), (64, 900, 8, 8, 96, 48, 2), (50, 1100, 8, 2, 48, 16, 16),
    (300, 300, 4, 4, 128, 16, 1)])
@pytest.mark.parametrize("drafts", [0, 3])
def test_batches_of_heads_beside_each_other(u, rows, length, heads, group, dim, page_tokens, blocks, dtype, drafts):
    lens = np.linspace(3, length, rows).astype(int)[np.random.default_rng(rows).permutation(rows)]
    lens[::17] = 0
    counts = None if drafts == 0 else 1 + np.arange(rows) % drafts
    c = segments(Case(rows, lens, counts, heads=heads, group=group, dim=dim, page_tokens=page_tokens, blocks=blocks,
                      dtype=dtype))
    for row in range(1, rows, 9):  # pages that are not there
        c.table[row, int(lens[row]) // page_tokens // 2] = -1 if row % 2 else c.pages
    worst = own_bound(c, call(u, c.gpu()))
    assert worst <= 1, worst


def test_outputs_beside_queries_and_over_them(u):
    """Queries and outputs in one tensor, every token's beside each other; outputs over queries are refused."""
    from u32_prefix_scan_gb300 import _native

    c = Case(31, [70, 45], [3, 2], heads=2, dim=64)
    d = c.gpu()
    want = call(u, d)
    both = torch.zeros(c.tokens, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    both[:, 0] = d["queries"]
    before = both[:, 0].clone()
    assert torch.equal(call(u, {**d, "queries": both[:, 0]}, out=both[:, 1]), want)
    assert torch.equal(both[:, 0], before)
    for out in (d["queries"], both.flatten(1, 2)[:, 1:5], both.flatten(1, 2)[:, :4]):
        queries = d["queries"] if out is d["queries"] else both[:, 0]
        with pytest.raises(_native.U32ScanError):
            call(u, {**d, "queries": queries}, out=out)
    assert torch.equal(both[:, 0], before) and torch.equal(both[:, 1], want)
