"""Pins of the oracle's logit rules, cache writes and attention (no GPU):
against numpy and torch on the CPU, written apart from the oracle; and the
refusals of the C entry points, which are decided on the host."""

import ctypes

import numpy as np
import pytest

import oracle
from u32_prefix_scan_gb300 import _native

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from u32_prefix_scan_gb300 import build

    build.build()
    return _native.lib()


# -- the rules on logits ----------------------------------------------------
def test_rules_by_hand():
    x = np.array([[2.0, -2.0, 4.0, 1.0, 0.5, 8.0]], np.float32)
    out, touched = oracle.adjust_logits(
        x, history=np.array([[0, 1, 2, 2, 9, -1]], np.int32), prompt_lens=[1], repetition=[2.0], presence=[0.25],
        frequency=[0.5], bias_tokens=np.array([[3, 3, 7]], np.int32), bias=np.array([[5.0, -1.0, 9.0]], np.float32),
        allowed=np.array([[0b011111]], np.uint32))
    # 0: prompt only; 1: once; 2: twice; 3: the later bias; 4: untouched; 5: not allowed
    assert out.tolist() == [[1.0, -4.0 - 0.75, 2.0 - 1.25, 0.0, 0.5, -np.inf]]
    assert touched.tolist() == [[True, True, True, True, False, True]]


@pytest.mark.parametrize("seed", range(4))
def test_rules_against_counts(seed):
    rng = np.random.default_rng(seed)
    rows, vocab, width = 3, 50, 80
    x = rng.standard_normal((rows, vocab)).astype(np.float32)
    h = rng.integers(0, vocab, (rows, width)).astype(np.int32)
    n, p = rng.integers(0, width + 1, rows), rng.integers(0, width + 1, rows)
    r, f, a = (rng.uniform(0.5, 1.5, rows).astype(np.float32) for _ in range(3))
    out, touched = oracle.adjust_logits(x, h, n, p, r, f, a)
    for b in range(rows):
        seen = np.bincount(h[b, : n[b]], minlength=vocab)
        made = np.bincount(h[b, min(p[b], n[b]) : n[b]], minlength=vocab)
        y = np.where(seen > 0, np.where(x[b] > 0, x[b] / r[b], x[b] * r[b]), x[b])
        y = np.where(made > 0, y - a[b] * made.astype(np.float32) - f[b], y)
        assert np.array_equal(out[b], y) and np.array_equal(touched[b], seen > 0)


@pytest.mark.parametrize("r", [0.0, -1.0, np.nan, np.inf])
def test_penalties_that_are_none(r):
    x = np.array([[1.5, -0.0, np.nan, -np.inf]], np.float32)
    out, _ = oracle.adjust_logits(x, history=[[0, 1, 2, 3]], repetition=[r], presence=[np.nan], frequency=[np.inf])
    assert np.array_equal(out, x, equal_nan=True)


# -- 8-bit codes and blocks -------------------------------------------------
def test_codes_are_e4m3():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(oracle.code_values(codes), want, equal_nan=True)
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(4000) * np.exp2(rng.uniform(-13, 8, 4000))).clip(-448, 448).astype(np.float32)
    mid = (oracle.code_values(codes[:126]) + oracle.code_values(codes[1:127])) / 2  # ties
    x = np.concatenate([x, mid, -mid, [0.0, -0.0, 448.0]]).astype(np.float32)
    assert np.array_equal(oracle.value_codes(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert oracle.value_codes([449.0, -1e30, np.inf, -np.inf]).tolist() == [0x7E, 0xFE, 0x7E, 0xFE]
    assert oracle.value_codes([np.nan]).tolist() == [0x7F]


def cache(pages, page_tokens, heads, dim, blocks):
    codes = np.zeros((2, pages, page_tokens, heads, dim), np.uint8)
    scales = np.zeros((2, pages, blocks, heads), np.float32)
    return codes[0], codes[1], scales[0], scales[1]


def test_a_scale_is_the_least_power_that_fits():
    k, v, ks, vs = cache(1, 4, 1, 2, 1)
    table = np.zeros((1, 1), np.int32)
    for top, want in ((448.0, 1.0), (np.nextafter(np.float32(448), np.float32(500)), 2.0), (0.25, 2.0**-10),
                      (7.0, 2.0**-6), (0.0, 2.0**-100), (np.inf, 2.0**-100), (3e38, 2.0**120)):
        x = np.array([[[top, 0.0]]], np.float32)
        _, _, got, _, _ = oracle.pages_append(k, v, table, [1], x, x, key_scales=ks, value_scales=vs)
        assert got[0, 0, 0] == want, top


@pytest.mark.parametrize("seed", range(3))
def test_appending_in_parts(seed):
    """Tokens written in any parts: what the cache holds is each value to half a
    step of the final scale, or of the scales on the way (powers of two:
    a code is rounded again only below its type's normal range)."""
    rng = np.random.default_rng(seed)
    n, dim = 37, 8
    x = (rng.standard_normal((n, 2, dim)) * np.exp2(rng.integers(-3, 4, (n, 1, 1)))).astype(np.float32)
    k, v, ks, vs = cache(12, 8, 2, dim, 2)
    table = rng.permutation(12)[:5].astype(np.int32)[None]
    at = 0
    while at < n:
        m = min(int(rng.integers(1, 9)), n - at)
        k, v, ks, vs, _ = oracle.pages_append(k, v, table, [at + m], x[at : at + m], -x[at : at + m], [0, m],
                                              key_scales=ks, value_scales=vs)
        at += m
    for t in range(n):
        p, slot = table[0, t // 8], t % 8
        for codes, scales, sign in ((k, ks, 1), (v, vs, -1)):
            s = scales[p, slot // 4]
            got = oracle.code_values(codes[p, slot]).astype(np.float64) * s[:, None]
            want = sign * x[t].astype(np.float64)
            # half a step: 2^-4 of the value, or of the least normal (2^-6 of the scale); once more for each of 3 later tokens
            assert np.all(np.abs(got - want) <= 2.0**-4 * np.abs(want) + 4 * 2.0**-10 * s[:, None])
            first, last = t - t % 4, min(t - t % 4 + 4, n)
            top = np.abs(x[first:last]).max((0, 2))
            assert np.all(top <= 448 * s) and np.all(top > 224 * s)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 10)).astype(np.float32)
    a = rng.uniform(0, 7, 4)
    y = oracle.rotate_heads(x, np.cos(a), np.sin(a), interleaved)
    i, j = (np.arange(0, 8, 2), np.arange(1, 8, 2)) if interleaved else (np.arange(4), np.arange(4, 8))
    z = (x[:, i] + 1j * x[:, j]) * np.exp(1j * a)
    # cosine and sine to half a step, two products and a sum
    assert np.allclose(y[:, i], z.real, rtol=0, atol=4 * 2.0**-24 * np.abs(z).max() * 2)
    assert np.allclose(y[:, j], z.imag, rtol=0, atol=4 * 2.0**-24 * np.abs(z).max() * 2)
    assert np.array_equal(y[:, 8:], x[:, 8:])


def test_what_is_not_written():
    k, v, ks, vs = (np.zeros((3, 2, 1, 2), np.float32) for _ in range(2)), None, None, None
    keys, values = k
    x = np.ones((6, 1, 2), np.float32)
    q = np.full((6, 1, 2), 2.0, np.float32)
    cos, sin = np.ones((3, 1)), np.zeros((3, 1))
    got = oracle.pages_append(keys, values, [[0, 5], [1, 2], [2, 1]], [4, 1, 2], x, x, starts=[0, 2, 4, 5],
                              status=[0, 1, -1], cos=cos, sin=sin, queries=q, queries_out=np.zeros_like(q))
    # row 0: positions 2, 3 on a page that is none; row 1: positions -1, 0; row 2: not served
    assert got[0][1, 0].tolist() == [[1.0, 1.0]] and got[0].sum() == 2
    # position 3 and -1 have no angles; token 5 is behind the last row's
    assert np.isnan(got[4][:, 0, 0]).tolist() == [False, True, True, False, False, False]
    assert got[4][5].tolist() == [[0.0, 0.0]]


# -- attention --------------------------------------------------------------
@pytest.mark.parametrize("counts", [None, [3, 1, 0, 2]])
def test_attention_is_the_softmax(counts):
    rng = np.random.default_rng(2)
    lens, heads, group, dim, pt = [9, 1, 0, 14], 2, 3, 4, 3
    pages = 12
    table = rng.permutation(pages)[:12].reshape(4, 3).astype(np.int32)
    table = np.concatenate([table, rng.permutation(pages)[:8].reshape(4, 2).astype(np.int32)], 1)
    codes = rng.integers(0, 0x70, (2, pages, pt, heads, dim)).astype(np.uint8)
    scales = rng.uniform(0.01, 0.1, (2, pages, 3, heads)).astype(np.float32)
    starts = None if counts is None else np.concatenate([[0], np.cumsum(counts)])
    tokens = 4 if counts is None else 6
    q = rng.standard_normal((tokens, heads * group, dim))
    got = oracle.pages_attend(q, codes[0], codes[1], scales[0], scales[1], table, lens, starts, 0.7)
    k, v = (torch.from_numpy(oracle.code_values(codes[i]).astype(np.float64) * scales[i][..., None]) for i in (0, 1))
    begin = 0
    for s, n in enumerate(lens):
        new = 1 if counts is None else counts[s]
        kk, vv = (t[torch.from_numpy(table[s]).long()].flatten(0, 1)[:n] for t in (k, v))
        for i in range(new):
            seen = n - new + i + 1
            for h in range(heads * group):
                if seen <= 0:
                    assert not got[begin + i, h].any()
                    continue
                w = torch.softmax(0.7 * (kk[:seen, h // group] @ torch.from_numpy(q[begin + i, h])), 0)
                assert np.allclose(got[begin + i, h], (w @ vv[:seen, h // group]).numpy(), rtol=1e-12, atol=1e-12)
        begin += new


# -- refusals of the C calls ------------------------------------------------
FAKE = 0x10000  # never dereferenced: every case fails a host check first


def rules(**kw):
    r = _native.LogitRulesStruct()
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_adjust_rejects_bad_arguments_on_host(lib):
    def call(logits=FAKE, type=0, rows=4, vocab=100, stride=100, out=FAKE + (1 << 20), out_stride=100, **kw):
        return lib.adjust_logits(logits, type, rows, vocab, stride, out, out_stride, ctypes.byref(rules(**kw)), None)

    for kw in (dict(type=3), dict(type=-1), dict(logits=None), dict(out=None), dict(logits=FAKE + 2), dict(out=FAKE + 1),
               dict(type=1, logits=FAKE + 1), dict(rows=1 << 28), dict(vocab=(1 << 22) + 1, out_stride=1 << 23),
               dict(stride=1 << 32), dict(out_stride=99), dict(out_stride=1 << 32), dict(out=FAKE + 4),
               dict(out=FAKE + 1200), dict(out=FAKE, stride=101), dict(history_width=5), dict(biases=3),
               dict(biases=3, bias=FAKE), dict(biases=3, bias_tokens=FAKE), dict(biases=1 << 31, bias=FAKE, bias_tokens=FAKE),
               dict(history=FAKE, history_width=1 << 31), dict(history=FAKE + 2, history_width=4),
               dict(history=FAKE, history_width=4, history_stride=1 << 32), dict(allowed=FAKE + 1),
               dict(allowed=FAKE, allowed_stride=1 << 32), dict(presence=FAKE + 3), dict(prompt_lens=FAKE + 2)):
        assert call(**kw) == _native.EINVAL, kw
    assert lib.adjust_logits(FAKE, 0, 4, 100, 100, FAKE + (1 << 20), 100, None, None) == _native.EINVAL
    assert call(rows=0, logits=None, out=None) == _native.OK
    assert call(vocab=0, logits=None, out=None) == _native.OK


def kv(**kw):
    c = _native.KVCacheStruct(FAKE, FAKE, _native.E4M3, 10, 16, 2, 64, 16 * 128, 128, 64, FAKE, FAKE, 2, 4)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def new_tokens(**kw):
    t = _native.NewTokensStruct(8, _native.BF16, FAKE, 128, 64, FAKE, 128, 64, FAKE, 4, 256, 64, FAKE, 256, 64, FAKE,
                                FAKE, 100, 32, 0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


BAD_ROWS = [dict(table=None), dict(table=FAKE + 2), dict(stride=3), dict(stride=1 << 31), dict(rows=1 << 31),
            dict(width=1 << 31, stride=1 << 31), dict(lens=None), dict(lens=FAKE + 1), dict(starts=FAKE + 2),
            dict(starts=None)]
BAD_CACHE = [dict(type=4), dict(type=-1), dict(pages=1 << 31), dict(page_tokens=0), dict(page_tokens=1 << 31),
             dict(heads=0), dict(heads=1 << 16), dict(dim=0), dict(dim=1025), dict(page_stride=1 << 40),
             dict(token_stride=1 << 40), dict(head_stride=1 << 40), dict(keys=None), dict(values=None),
             dict(key_scales=None), dict(value_scales=None), dict(blocks=0), dict(blocks=3), dict(key_scales=FAKE + 2),
             dict(scale_stride=1 << 40), dict(page_stride=0), dict(token_stride=0), dict(head_stride=0)]


def test_append_rejects_bad_arguments_on_host(lib):
    def call(cache=None, new=None, table=FAKE, stride=4, rows=3, width=4, lens=FAKE, starts=FAKE, status=None):
        return lib.pages_append(kv(**(cache or {})), table, stride, rows, width, lens, starts, status,
                                ctypes.byref(new_tokens(**(new or {}))), None)

    for kw in BAD_ROWS + [dict(status=FAKE + 1)]:
        assert call(**kw) == _native.EINVAL, kw
    for cache in BAD_CACHE + [dict(type=_native.F16), dict(type=_native.F32)]:
        assert call(cache=cache) == _native.EINVAL, cache
    for new in (dict(type=3), dict(type=-1), dict(tokens=1 << 31), dict(keys=None), dict(values=None),
                dict(queries_out=None), dict(keys=FAKE + 1), dict(values=FAKE + 1), dict(queries=FAKE + 1),
                dict(queries_out=FAKE + 1), dict(cos=None), dict(sin=None), dict(cos=FAKE + 2), dict(pairs=33),
                dict(positions=1 << 31), dict(key_head_stride=1 << 40), dict(out_token_stride=1 << 40),
                dict(q_heads=1 << 16)):
        assert call(new=new) == _native.EINVAL, new
    assert lib.pages_append(None, FAKE, 4, 3, 4, FAKE, FAKE, None, ctypes.byref(new_tokens()), None) == _native.EINVAL
    assert lib.pages_append(kv(), FAKE, 4, 3, 4, FAKE, FAKE, None, None, None) == _native.EINVAL
    assert call(new=dict(tokens=0)) == _native.OK
    assert call(rows=0, lens=None, table=None) == _native.OK


def test_attend_rejects_bad_arguments_on_host(lib):
    need = lib.u32scan_workspace_bytes(_native.OP_ATTEND, 8)
    assert need >= 256 and need % 256 == 0 and need == lib.u32scan_workspace_bytes(_native.OP_ATTEND, 1 << 20)

    def call(cache=None, table=FAKE, stride=4, rows=3, width=4, lens=FAKE, starts=FAKE, tokens=8, queries=FAKE,
             type=_native.BF16, q_heads=4, qs=256, qh=64, out=FAKE + (1 << 20), os=256, oh=64, ws=FAKE, ws_bytes=need):
        return lib.pages_attend(kv(**(cache or {})), table, stride, rows, width, lens, starts, tokens, queries, type,
                                q_heads, qs, qh, out, os, oh, 1.0, ws, ws_bytes, None)

    for kw in BAD_ROWS:
        assert call(**kw) == _native.EINVAL, kw
    for cache in BAD_CACHE + [dict(type=_native.BF16), dict(dim=72), dict(dim=272), dict(keys=FAKE + 8),
                              dict(values=FAKE + 8), dict(page_stride=16 * 128 + 8), dict(token_stride=136),
                              dict(head_stride=72)]:
        assert call(cache=cache) == _native.EINVAL, cache
    for kw in (dict(type=0), dict(type=3), dict(tokens=1 << 31), dict(queries=None), dict(out=None),
               dict(queries=FAKE + 8), dict(qs=260), dict(qh=68), dict(out=FAKE + 1), dict(q_heads=0), dict(q_heads=5),
               dict(q_heads=1 << 16), dict(qs=1 << 40), dict(oh=1 << 40), dict(tokens=1 << 30, q_heads=8)):
        assert call(**kw) == _native.EINVAL, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(ws_bytes=need - 256)):
        assert call(**kw) == _native.EWORKSPACE, kw
    assert call(tokens=0) == _native.OK
    assert call(rows=0, lens=None, table=None) == _native.OK


def shared(a, b):
    """Whether two arrays (first element, counts, strides, run) have an element in common."""
    places = []
    for at, counts, strides, run in (a, b):
        i = np.arange(at, at + run)
        for n, s in zip(counts, strides):
            i = (i[None] + np.arange(n)[:, None] * s).ravel()
        places.append(np.unique(i))
    return np.intersect1d(*places).size > 0


def attend_refuses(lib, tokens, q_heads, q, out):
    """Whether pages_attend refuses queries and out ((first element, token stride, head stride) of bf16, heads of 16
    elements), by what it says where both are sound but the workspace is missing."""
    cache = kv(dim=16, heads=1, head_stride=0, token_stride=16, page_stride=256)
    status = lib.pages_attend(cache, FAKE, 4, tokens, 4, FAKE, None, tokens, FAKE + 2 * q[0], _native.BF16, q_heads, *q[1:],
                              FAKE + 2 * out[0], *out[1:], 1.0, None, 0, None)
    assert status in (_native.EINVAL, _native.EWORKSPACE)
    return status == _native.EINVAL


def test_attend_refuses_an_output_that_shares_memory_with_the_queries(lib):
    for q, out, refused in (
            ((0, 64, 16), (0, 64, 16), True), ((0, 64, 16), (8, 64, 16), True), ((0, 64, 16), (64, 64, 16), True),
            ((0, 64, 16), (64 * 5, 64, 16), False), ((64 * 5, 64, 16), (0, 64, 16), False),
            ((64 * 5, 64, 16), (1, 64, 16), True), ((64 * 5 + 8, 64, 16), (1, 64, 16), False),
            ((0, 192, 16), (64, 192, 16), False), ((0, 192, 16), (128, 192, 16), False),  # parts of one row
            ((0, 192, 16), (56, 192, 16), True), ((0, 192, 48), (16, 192, 48), False), ((0, 192, 48), (9, 192, 48), True),
            ((0, 16, 80), (0, 64, 16), True), ((0, 0, 0), (0, 64, 16), True), ((0, 0, 0), (16, 64, 16), False)):
        assert attend_refuses(lib, 5, 4, q, out) == refused, (q, out)


@pytest.mark.parametrize("seed", range(3))
def test_shared_memory_is_found_exactly(lib, seed):
    rng, found = np.random.default_rng(seed), 0
    for _ in range(400):
        tokens, heads = (int(x) for x in rng.integers(1, 7, 2))
        q, out = ((int(rng.integers(0, 30)) * 8, int(rng.integers(0, 30)) * 8, int(rng.integers(0, 30)) * 8) for _ in range(2))
        if rng.random() < 0.5:
            out = (out[0], *q[1:])
        want = shared(*((x[0], (tokens, heads), x[1:], 16) for x in (q, out)))
        assert attend_refuses(lib, tokens, heads, q, out) == want, (tokens, heads, q, out)
        found += want
    assert 40 < found < 360


def test_shared_memory_of_the_largest_sizes(lib):
    """Strides and counts whose products pass 64 bits."""
    far = 1 << 39
    assert not attend_refuses(lib, (1 << 31) // 8 - 1, 8, (0, far, 16), (128, far, 16))
    assert attend_refuses(lib, (1 << 31) // 8 - 1, 8, (0, far, 16), (120, far, 16))
    assert attend_refuses(lib, (1 << 31) // 8 - 1, 8, (far * 1000, far, 16), (0, far, 16))


@pytest.mark.parametrize("type", [_native.F32, _native.BF16])
def test_append_refuses_rotated_queries_over_its_inputs(lib, type):
    """8 tokens of 4 heads of 64 elements, queries_out over a part of another array or over queries laid out otherwise."""
    size, far = 4 if type == _native.F32 else 2, 1 << 24
    apart = dict(type=type, keys=FAKE + far, values=FAKE + 2 * far, queries=FAKE + 3 * far, queries_out=FAKE + 4 * far)
    for name, at in (("keys", FAKE + far), ("values", FAKE + 2 * far), ("queries", FAKE + 3 * far)):
        for kw in (dict(queries_out=at + 64 * size), dict(queries_out=at - 63 * size),
                   dict(queries_out=at, out_token_stride=320), dict(queries_out=at, out_head_stride=512, out_token_stride=64),
                   dict(queries_out=at + (128 * 7 + 64) * size)):
            new = new_tokens(**{**apart, **kw})
            assert lib.pages_append(kv(type=type), FAKE, 4, 3, 4, FAKE, FAKE, None, ctypes.byref(new), None) == _native.EINVAL, (name, kw)
