"""GPU parity of pages_append against the CPU oracle, bit for bit: caches of
every type, rotations, blocks that grow, ragged rows, strides and pages in any
order."""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def u():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from u32_prefix_scan_gb300 import build

    build.build()
    import u32_prefix_scan_gb300 as u

    return u


def angles(positions, pairs):
    rate = 10000.0 ** (-np.arange(pairs) / max(pairs, 1))
    a = np.arange(positions)[:, None] * rate
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


class Case:
    """A cache, its rows and the new tokens, on the host."""

    def __init__(self, seed, lens, counts, *, heads=2, dim=16, page_tokens=4, blocks=2, dtype="bf16", cache="e4m3",
                 q_heads=0, pairs=None, interleaved=False, positions=None, spare=3, tail=0, one_each=False):
        rng = np.random.default_rng(seed)
        self.dtype, self.cache, self.interleaved = dtype, cache, interleaved
        self.lens, counts = np.asarray(lens, np.int32), np.asarray(counts)
        rows = len(lens)
        need = -(-np.maximum(self.lens, 0) // page_tokens)
        self.pages = int(need.sum()) + spare
        width = max(int(need.max(initial=0)), 1)
        place = rng.permutation(self.pages)
        self.table = np.full((rows, width), -1, np.int32)
        at = 0
        for s in range(rows):
            self.table[s, : need[s]] = place[at : at + need[s]]
            at += need[s]
        self.starts = None if one_each else np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.tokens = int(counts.sum()) + tail
        shape = (self.pages, page_tokens, heads, dim)

        def values(*shape):
            x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, shape[:-1] + (1,)))
            return torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])

        if cache == "e4m3":
            codes = rng.integers(0, 256, (2, *shape)).astype(np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x41
            self.keys, self.values = codes
            s = np.exp2(rng.integers(-9, 2, (2, self.pages, blocks, heads))).astype(np.float32)
            s[rng.random(s.shape) < 0.1] = 0.3  # a caller's own
            s[rng.random(s.shape) < 0.05] = 0.0
            s[rng.random(s.shape) < 0.05] = np.nan
            self.key_scales, self.value_scales = s
        else:
            self.keys, self.values = (values(*shape).float().numpy() for _ in range(2))
            self.key_scales = self.value_scales = None
        self.new_keys, self.new_values = values(self.tokens, heads, dim), values(self.tokens, heads, dim)
        self.queries = values(self.tokens, q_heads, dim) if q_heads else None
        self.cos = self.sin = None
        if pairs is None:
            pairs = dim // 2
        if pairs:
            self.cos, self.sin = angles(positions if positions is not None else int(self.lens.max(initial=0)) + 3, pairs)
        self.status = None

    def gpu(self):
        def dev(a):
            return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()

        d = {k: dev(getattr(self, k)) for k in ("table", "lens", "starts", "status", "cos", "sin", "key_scales",
                                                "value_scales")}
        for k in ("keys", "values"):
            t = dev(getattr(self, k))
            d[k] = t.view(torch.float8_e4m3fn) if self.cache == "e4m3" else t.to(TYPES[self.cache])
        for k in ("new_keys", "new_values", "queries"):
            t = getattr(self, k)
            d[k] = None if t is None else t.cuda()
        d["queries_out"] = None if self.queries is None else torch.full_like(d["queries"], 7.0)
        return d

    def want(self):
        q = None if self.queries is None else self.queries.float().numpy()
        with np.errstate(invalid="ignore", over="ignore"):
            return oracle.pages_append(
                self.keys, self.values, self.table, self.lens, self.new_keys.float().numpy(),
                self.new_values.float().numpy(), self.starts, self.status, self.cos, self.sin, self.interleaved,
                self.key_scales, self.value_scales, q, None if q is None else np.full_like(q, 7.0))

    def check(self, d):
        keys, values, ks, vs, q = self.want()
        for name, want, scales in (("keys", keys, ks), ("values", values, vs)):
            got = d[name]
            if self.cache == "e4m3":
                g = got.view(torch.uint8).cpu().numpy()
                nan = (g & 0x7F == 0x7F) & (want & 0x7F == 0x7F)
                assert np.array_equal(np.where(nan, 0, g), np.where(nan, 0, want)), name
                assert np.array_equal(d[name[:-1] + "_scales"].cpu().numpy(), scales, equal_nan=True), name + " scales"
            else:
                w = torch.from_numpy(want).to(TYPES[self.cache])
                assert torch.equal(got.cpu().nan_to_num(1234.0), w.nan_to_num(1234.0)), name
        if q is not None:
            w = torch.from_numpy(q).to(TYPES[self.dtype])
            got = d["queries_out"].cpu()
            assert torch.equal(got.isnan(), w.isnan()) and torch.equal(got.nan_to_num(0.5), w.nan_to_num(0.5))


def call(u, d, cache=None, **kw):
    cache = cache or u.KVCache(d["keys"], d["values"], d["key_scales"], d["value_scales"])
    args = {k: d[k] for k in ("starts", "status", "cos", "sin", "queries", "queries_out")}
    out = u.pages_append(cache, d["table"], d["lens"], d["new_keys"], d["new_values"], **{**args, **kw})
    torch.cuda.synchronize()
    return out


CACHES = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "e4m3"), ("f16", "e4m3"), ("bf16", "e4m3")]


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,pairs", [(16, 8), (16, 3), (64, 32), (128, 64), (80, 20), (7, 3), (2, 1), (256, 128), (33, 0)])
def test_types_and_rotations(u, dtype, cache, interleaved, dim, pairs):
    c = Case(dim + pairs, [5, 9, 1, 12], [3, 4, 1, 12], dim=dim, pairs=pairs, interleaved=interleaved, dtype=dtype,
             cache=cache, q_heads=3)
    d = c.gpu()
    call(u, d, interleaved=interleaved)
    c.check(d)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page_tokens,blocks", [(1, 1), (4, 4), (6, 2), (16, 1), (20, 2), (48, 2), (128, 2)])
@pytest.mark.parametrize("lens,counts", [([1], [1]), ([130, 7, 64], [130, 7, 64]), ([131, 200, 5], [1, 70, 0]),
                                         ([0, 3, 0, 50], [0, 1, 0, 49])])
def test_pages_and_blocks(u, cache, page_tokens, blocks, lens, counts):
    c = Case(page_tokens, lens, counts, page_tokens=page_tokens, blocks=blocks, cache=cache, q_heads=2, heads=3)
    d = c.gpu()
    call(u, d)
    c.check(d)


@pytest.mark.parametrize("rows", [1, 2, 64, 300])
def test_one_token_a_row(u, rows):
    lens = 1 + np.arange(rows) * 7 % 40
    c = Case(rows, lens, np.ones(rows, int), one_each=True, dim=64, q_heads=8, heads=2, page_tokens=16, blocks=2)
    d = c.gpu()
    call(u, d)
    c.check(d)


def test_tokens_one_by_one_are_the_oracles(u):
    """A block filled token by token: its scale grows with its largest, the
    older codes are rounded each time."""
    c = Case(5, [8], [8], dim=32, page_tokens=8, blocks=1, pairs=0, dtype="f32")
    c.new_keys *= torch.exp2(torch.arange(8.0))[:, None, None]  # grows, so every token raises it
    c.new_values *= torch.exp2(-torch.arange(8.0))[:, None, None]
    d = c.gpu()
    cache = u.KVCache(d["keys"], d["values"], d["key_scales"], d["value_scales"])
    state = (c.keys, c.values, c.key_scales, c.value_scales)
    for t in range(8):
        lens = np.array([t + 1], np.int32)
        u.pages_append(cache, d["table"], torch.from_numpy(lens).cuda(), d["new_keys"][t : t + 1], d["new_values"][t : t + 1])
        state = oracle.pages_append(state[0], state[1], c.table, lens, c.new_keys[t : t + 1].numpy(),
                                    c.new_values[t : t + 1].numpy(), key_scales=state[2], value_scales=state[3])[:4]
    assert np.array_equal(d["keys"].view(torch.uint8).cpu().numpy(), state[0])
    assert np.array_equal(d["values"].view(torch.uint8).cpu().numpy(), state[1])
    assert np.array_equal(d["key_scales"].cpu().numpy(), state[2], equal_nan=True)
    assert np.array_equal(d["value_scales"].cpu().numpy(), state[3], equal_nan=True)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_what_is_not_written(u, cache):
    """Rows that were not served, tokens past the table, the pool or the
    angles, rows longer than they say, tokens behind the last row's."""
    c = Case(3, [9, 14, 6, 3, 20], [4, 9, 2, 5, 7], cache=cache, dtype="f16", q_heads=2, tail=6, positions=17)
    c.status = np.array([0, 1, -2, 0, 3], np.int32)
    c.table[1, 1], c.table[1, 2] = -1, c.pages
    c.lens[0] += 40  # past the table's width
    d = c.gpu()
    call(u, d)
    c.check(d)
    assert torch.all(d["queries_out"][c.tokens - 6 :] == 7)


@pytest.mark.parametrize("starts", [[0, 5, 2, 8], [-3, 2, 40, 41], [2, 3, 4, 5], [9, 9, 9, 9]])
def test_starts_out_of_order_stay_in_bounds(u, starts):
    """The written tokens are unspecified, what no row names stays."""
    c = Case(8, [4, 7, 9], [2, 3, 4], q_heads=1)
    c.starts = np.array(starts, np.int32)
    d = c.gpu()
    call(u, d)
    free = np.setdiff1d(np.arange(c.pages), c.table)
    assert np.array_equal(d["keys"].view(torch.uint8).cpu().numpy()[free], c.keys[free])


@pytest.mark.parametrize("kind", ["zero", "nan", "inf", "tiny", "huge"])
def test_special_values(u, kind):
    c = Case(11, [6, 11], [6, 4], dtype="f32", dim=32, pairs=0, page_tokens=4, blocks=1)
    x = c.new_keys
    if kind == "zero":
        x.zero_()
    elif kind == "nan":
        x[::2, :, 3] = float("nan")
    elif kind == "inf":
        x[1::2, :, 5] = float("inf")
        x[0] = -float("inf")
    elif kind == "tiny":
        x *= 2.0**-140
    else:
        x *= 2.0**120
    d = c.gpu()
    call(u, d)
    c.check(d)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_strides(u, cache, offset):
    """Keys, values and queries cut out of one projection; heads before
    tokens within a page; pages with room between them; odd addresses."""
    c = Case(21, [30, 17, 9], [13, 17, 1], cache=cache, heads=3, dim=32, q_heads=5, page_tokens=8, blocks=2)
    d = c.gpu()
    fused = torch.zeros(c.tokens, 11 * 32 + offset, dtype=torch.bfloat16, device="cuda")
    heads = fused[:, offset:].unflatten(1, (11, 32))
    for k, at, n in (("queries", 0, 5), ("new_keys", 5, 3), ("new_values", 8, 3)):
        heads[:, at : at + n] = d[k]
        d[k] = heads[:, at : at + n]
    for k in ("keys", "values"):
        t = d[k]
        item = t.element_size()
        room = torch.zeros(c.pages, (3 * 8 * 32 + 64) * item, dtype=torch.uint8, device="cuda")
        part = room[:, offset * item : (offset + 3 * 8 * 32) * item]
        view = part.view(t.dtype).unflatten(1, (3, 8, 32)).transpose(1, 2)
        view.view(torch.uint8).copy_(t.view(torch.uint8))
        d[k] = view
    out = torch.full((c.tokens, 5, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    d["queries_out"] = out[:, :, offset : offset + 32]
    call(u, d)
    c.check({**d, "keys": d["keys"].contiguous(), "values": d["values"].contiguous()})
    assert torch.all(out[:, :, :offset] == 7) and torch.all(out[:, :, offset + 32 :] == 7)


def test_queries_in_place_and_again(u):
    c = Case(31, [30, 17], [13, 17], dim=64, q_heads=5, page_tokens=8, blocks=2)
    d = c.gpu()
    d["queries_out"] = d["queries"]
    assert call(u, d) is d["queries"]
    keys, ks = d["keys"].view(torch.uint8).clone(), d["key_scales"].clone()
    c.check(d)
    # the same tokens again change nothing more
    call(u, d, queries=None, queries_out=None)
    assert torch.equal(d["keys"].view(torch.uint8), keys)
    assert torch.equal(d["key_scales"].nan_to_num(5.0), ks.nan_to_num(5.0))


def test_none_of_it(u):
    c = Case(1, [3], [1], one_each=True)
    d = c.gpu()
    before = d["keys"].view(torch.uint8).clone()
    cache = u.KVCache(d["keys"], d["values"], d["key_scales"], d["value_scales"])
    none = d["new_keys"][:0]
    u.pages_append(cache, d["table"][:0], d["lens"][:0], none, none)
    u.pages_append(cache, d["table"], d["lens"], none, none, starts=torch.zeros(2, dtype=torch.int32, device="cuda"))
    empty = u.KVCache(d["keys"][:0], d["values"][:0], d["key_scales"][:0], d["value_scales"][:0])
    u.pages_append(empty, d["table"], d["lens"], d["new_keys"], d["new_values"])
    torch.cuda.synchronize()
    assert torch.equal(d["keys"].view(torch.uint8), before)


def test_another_stream_and_a_graph(u):
    c = Case(41, [30, 17, 9], [1, 1, 1], one_each=True, dim=64, q_heads=4, page_tokens=8, blocks=1)
    d = c.gpu()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(u, d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    c.check(d)
    d = c.gpu()
    cache = u.KVCache(d["keys"], d["values"], d["key_scales"], d["value_scales"])
    start = {k: d[k].clone() for k in ("keys", "values", "key_scales", "value_scales")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call_only = {k: d[k] for k in ("cos", "sin", "queries", "queries_out")}
        u.pages_append(cache, d["table"], d["lens"], d["new_keys"], d["new_values"], **call_only)
    for seed in (1, 2):
        fresh = Case(41, [30, 17, 9], [1, 1, 1], one_each=True, dim=64, q_heads=4, page_tokens=8, blocks=1)
        fresh.new_keys, fresh.lens = fresh.new_keys * seed, fresh.lens - seed
        d["new_keys"].copy_(fresh.new_keys)
        d["lens"].copy_(torch.from_numpy(fresh.lens))
        for k, t in start.items():
            d[k].view(torch.uint8).copy_(t.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        fresh.check(d)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_offsets_past_32_bits(u, cache):
    """Pages half a gigabyte apart."""
    c = Case(51, [30, 41], [13, 41], cache=cache, heads=2, dim=32, page_tokens=8, blocks=2)
    d = c.gpu()
    room = torch.empty(c.pages << 29, dtype=torch.uint8, device="cuda").view(c.pages, 1 << 29)
    assert room.numel() > 1 << 32
    for at, k in ((0, "keys"), (1 << 28, "values")):
        t = d[k]
        size = 8 * 2 * 32 * t.element_size()
        view = room[:, at : at + size].view(t.dtype).view(c.pages, 8, 2, 32)
        view.view(torch.uint8).copy_(t.view(torch.uint8))
        d[k] = view
    call(u, d)
    c.check({**d, "keys": d["keys"].contiguous(), "values": d["values"].contiguous()})


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("dim,heads,q_heads,page_tokens,blocks", [(64, 2, 6, 16, 1), (128, 1, 2, 48, 2)])
def test_many_tokens(u, dtype, cache, dim, heads, q_heads, page_tokens, blocks):
    """More tokens than blocks of 64 threads run at a time."""
    c = Case(dim, [900, 1500, 17, 3, 400], [700, 1500, 1, 0, 300], dim=dim, dtype=dtype, cache=cache, heads=heads, q_heads=q_heads,
             page_tokens=page_tokens, blocks=blocks, tail=5)
    assert c.tokens > 2432
    d = c.gpu()
    call(u, d)
    c.check(d)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,most", [(32, 3), (33, 2), (100, 5), (1025, 2), (1500, 3)])
def test_many_rows_of_any_number_of_tokens(u, cache, rows, most):
    """Rows found among more than 32 and more than 32 * 32, empty ones beside each other among them."""
    rng = np.random.default_rng(rows)
    counts = rng.integers(0, most + 1, rows)
    counts[rows // 3 : rows // 3 + 40] = 0
    counts[[0, -1]] = [0, 1]
    lens = counts + rng.integers(0, 20, rows)
    c = Case(rows, lens, counts, dim=16, heads=1, q_heads=2, page_tokens=8, blocks=2, cache=cache, tail=2)
    d = c.gpu()
    call(u, d)
    c.check(d)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_rotated_queries_beside_the_inputs_and_over_them(u, cache):
    """Queries, keys and values cut out of one projection, queries rotated in place in it or into a
    part of it of their own; over keys, values or other queries they are refused."""
    from u32_prefix_scan_gb300 import _native

    c = Case(61, [30, 17, 9], [13, 17, 1], cache=cache, heads=3, dim=32, q_heads=5, page_tokens=8, blocks=2)
    for place in ("in place", "beside"):
        d = c.gpu()
        fused = torch.zeros(c.tokens, 16, 32, dtype=torch.bfloat16, device="cuda")
        for k, at, n in (("queries", 0, 5), ("new_keys", 5, 3), ("new_values", 8, 3)):
            fused[:, at : at + n] = d[k]
            d[k] = fused[:, at : at + n]
        if place == "in place":
            d["queries_out"] = d["queries"]
        else:
            d["queries_out"] = fused[:, 11:].fill_(7.0)
        before = fused.clone()
        for out in (fused[:, 1:6], fused[:, 5:10], fused[:, 6:11], fused[:, 4:9]):
            with pytest.raises(_native.U32ScanError):
                call(u, d, queries_out=out)
        assert torch.equal(fused, before)
        call(u, d)
        c.check(d)
