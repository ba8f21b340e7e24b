"""Pins of the oracle's token sampler and paged-cache operations (no GPU):
against softmax in 64 bits, against numpy sorts written apart from the
oracle, and against a cache's own invariants; and the refusals of the C
entry points, which are decided on the host."""

import ctypes

import numpy as np
import pytest

import oracle
from u32_prefix_scan_gb300 import _native, inputs


@pytest.fixture(scope="module")
def lib():
    from u32_prefix_scan_gb300 import build

    build.build()
    return _native.lib()


# A weight's relative error: y = (m - l) * scale < 32 carries three roundings
# (1.5 ulp of at most 2^-19, times ln 2) and 2^-y 1.9e-7 more; its floor is
# off by at most 2^-31 of the largest weight.
REL = 1.5 * 2.0**-19 * np.log(2.0) + 2e-7
ABS = 2.0**-31


def softmax64(x, t):
    z = (x.astype(np.float64) - x.max()) / t
    w = np.exp(z)
    return w / w.sum(), w


@pytest.mark.parametrize("t", [0.3, 1.0, 2.5])
@pytest.mark.parametrize("n", [1, 2, 37, 4001])
def test_probabilities_are_the_softmax(t, n):
    rng = np.random.default_rng(n)
    x = (3 * rng.standard_normal(n)).astype(np.float32)
    p, w = softmax64(x, t)
    words = inputs.splitmix_u32(3, 0, 200)
    tok, prob = oracle.sample_tokens(np.tile(x, (200, 1)), words, temperature=np.full(200, t, np.float32))
    rel = 2 * REL + n * ABS  # of the weight and of the sum
    # and the probability's own rounding to float
    assert np.all(np.abs(prob - p[tok]) <= p[tok] * (rel + 2.0**-24) + ABS)


def test_draw_covers_the_distribution():
    """With words spread evenly over [0, 2^32) every token comes up in
    proportion to its probability, to within one word."""
    x = np.log(np.array([[1, 2, 3, 4, 6]], dtype=np.float32))
    words = (np.arange(4096, dtype=np.uint64) << np.uint64(20)).astype(np.uint32)
    tok, prob = oracle.sample_tokens(np.repeat(x, 4096, 0), words)
    assert np.all(np.diff(tok) >= 0)  # index order
    counts = np.bincount(tok, minlength=5)
    assert np.all(np.abs(counts - 4096 * np.array([1, 2, 3, 4, 6]) / 16) <= 1)
    assert oracle.sample_tokens(x, [0])[0][0] == 0 and oracle.sample_tokens(x, [0xFFFFFFFF])[0][0] == 4


@pytest.mark.parametrize("k", [1, 2, 5, 39, 40, 1000])
def test_top_k_keeps_the_k_largest_lowest_index_first(k):
    rng = np.random.default_rng(k)
    x = rng.integers(-4, 5, 40).astype(np.float32)  # many ties
    order = sorted(range(40), key=lambda i: (-x[i], i))
    keep = set(order[:k])
    words = inputs.splitmix_u32(4, 0, 400)
    tok, prob = oracle.sample_tokens(np.tile(x, (400, 1)), words, top_k=np.full(400, k))
    w = np.exp(x.astype(np.float64))
    total = sum(w[i] for i in keep)
    assert set(tok) <= keep
    assert np.allclose(prob, w[tok] / total, rtol=1e-5, atol=0)


@pytest.mark.parametrize("p", [1e-6, 0.3, 0.5, 0.9, 0.999])
def test_top_p_keeps_the_shortest_prefix(p):
    x = np.log(np.array([2, 16, 1, 8, 4, 1], dtype=np.float32))
    share = np.array([2, 16, 1, 8, 4, 1]) / 32.0
    order = [1, 3, 4, 0, 2, 5]
    keep, mass = [], 0.0
    for i in order:
        if mass >= p:
            break
        keep.append(i)
        mass += share[i]
    tok, prob = oracle.sample_tokens(np.tile(x, (300, 1)), inputs.splitmix_u32(5, 0, 300),
                                     top_p=np.full(300, p, np.float32))
    assert set(tok) <= set(keep)
    assert np.allclose(prob, share[tok] / share[keep].sum(), rtol=1e-5, atol=0)


def test_min_p_and_special_values():
    inf, nan = np.float32("inf"), np.float32("nan")
    low = np.finfo(np.float32).min
    x = np.log(np.array([[1, 8, 4, 2]], dtype=np.float32))
    tok, prob = oracle.sample_tokens(np.repeat(x, 200, 0), inputs.splitmix_u32(6, 0, 200),
                                     min_p=np.full(200, 0.4, np.float32))
    assert set(tok) == {1, 2} and np.allclose(prob, np.array([0, 8, 4, 0])[tok] / 12, rtol=1e-5)
    rows = np.array([[-inf, nan, -inf], [nan, 1, nan], [inf, 0, inf], [low, low, 0], [low, low, low], [-0.0, 0, -0.0]],
                    dtype=np.float32)
    tok, prob = oracle.sample_tokens(rows, [0xFFFFFFFF] * 6)
    assert tok.tolist() == [-1, 1, 2, 2, 2, 2]
    assert np.allclose(prob, [0, 1, 0.5, 1, 1 / 3, 1 / 3])
    tok, prob = oracle.sample_tokens(rows, [0xFFFFFFFF] * 6, temperature=[0.0] * 6)
    assert tok.tolist() == [-1, 1, 0, 2, 0, 0] and prob.tolist() == [0, 1, 1, 1, 1, 1]


def make_cache(seed, rows, width, pages, page_tokens, empty_from=None):
    """A consistent random cache in which odd rows share the front of the
    row before them."""
    rng = np.random.default_rng(seed)
    table = np.full((rows, width), -1, np.int32)
    lens = np.zeros(rows, np.int32)
    free = list(rng.permutation(pages))
    for s in range(rows if empty_from is None else empty_from):
        length = int(rng.integers(0, width * page_tokens + 1))
        n = -(-length // page_tokens)
        share = 0
        if s % 2 and table[s - 1, 0] >= 0:
            share = int(rng.integers(0, min(n, lens[s - 1] // page_tokens, length // page_tokens) + 1))
        if n - share > len(free):
            continue
        table[s, :share] = table[s - 1, :share]
        table[s, share:n] = [free.pop() for _ in range(n - share)]
        lens[s] = length
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    return table, lens, refs


def check_cache(table, lens, refs, page_tokens):
    """refs count the entries in use."""
    used = np.arange(table.shape[1])[None, :] < -(-lens // page_tokens)[:, None]
    assert np.array_equal(np.bincount(table[used], minlength=refs.size), refs)


def read_row(pool, table, lens, s, page_tokens):
    """A row's bytes, token by token (a page holds its tokens one after another)."""
    n = -(-int(lens[s]) // page_tokens)
    pages = pool[:, table[s, :n]]
    planes = pool.shape[0]
    per = pool.shape[2] // page_tokens
    return pages.reshape(planes, -1, per)[:, : int(lens[s])]


@pytest.mark.parametrize("page_tokens", [1, 4, 7])
def test_a_cache_keeps_its_rows(page_tokens):
    rows, width, pages = 24, 6, 90
    rng = np.random.default_rng(page_tokens)
    table, lens, refs = make_cache(1, rows, width, pages, page_tokens, empty_from=12)
    pool = rng.integers(0, 256, (2, pages, 3 * page_tokens), dtype=np.uint8)
    was = [read_row(pool, table, lens, s, page_tokens) for s in range(rows)]
    parent = np.full(rows, -1, np.int32)
    parent[12:] = rng.integers(0, 12, 12)
    grow = rng.integers(0, 3, rows).astype(np.int32)
    before = (refs == 0).sum()
    t, l, r, status, left, p = oracle.pages_fork(table, lens, refs, page_tokens, parent, grow, pool)
    assert (status >= 0).any() and left == before - status[status > 0].sum() == (r == 0).sum()
    check_cache(t, l, r, page_tokens)
    for s in range(rows):
        src = parent[s] if parent[s] >= 0 else s
        if status[s] >= 0:
            assert l[s] == lens[src] + grow[s]
            got = read_row(p, t, l, s, page_tokens)
            assert np.array_equal(got[:, : lens[src]], was[src])
        else:
            assert l[s] == lens[s] and np.array_equal(t[s], table[s])
    release = (rng.random(rows) < 0.5).astype(np.int32)
    held = [read_row(p, t, l, s, page_tokens) for s in range(rows)]
    free_before = (r == 0).sum()
    t, l, r, freed = oracle.pages_free(t, l, r, page_tokens, release)
    assert freed == (r == 0).sum() - free_before
    check_cache(t, l, r, page_tokens)
    t, r, live, remap, p = oracle.pages_compact(t, l, r, page_tokens, p)
    assert live == (r != 0).sum() and np.all(r[:live] != 0) and np.all(r[live:] == 0)
    check_cache(t, l, r, page_tokens)
    for s in range(rows):
        if release[s]:
            assert l[s] == 0
        else:
            assert np.array_equal(read_row(p, t, l, s, page_tokens), held[s])


def test_fork_refusals_and_running_out():
    table = np.array([[0, 1, 2], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1], [3, -1, -1]], np.int32)
    lens = np.array([9, 0, 0, 0, 4], np.int32)
    refs = np.array([1, 1, 1, 1, 0, 0], np.int32)
    run = lambda parent, grow: oracle.pages_fork(table, lens, refs, 4, parent, grow)[3].tolist()  # noqa: E731
    assert run([-1, 0, 0, 0, -1], [0, 0, 0, 0, 0]) == [0, 1, 1, -2, 0]  # two pages for three children
    assert run([-1, 1, 7, 4, 0], [0, 0, 0, 0, 0]) == [0, -1, -1, -1, -1]  # itself, no row, a child, not empty
    assert run([-1, -1, -1, -1, -1], [4, 0, 0, 0, 1]) == [-1, 0, 0, 0, 1]  # too long
    assert run(None, [-1, 0, 0, 0, 9]) == [-1, 0, 0, 0, -1]
    assert run(None, [3, 9, 0, 0, 4]) == [0, -2, 0, 0, -2]  # a later row does not overtake


# --------------------------------------------------------------------------
# refusals of the C entry points (nothing is dereferenced or launched)
# --------------------------------------------------------------------------
FAKE = 0x10000


def sample_call(lib, **kw):
    a = dict(logits=FAKE, type=_native.F32, rows=4, vocab=100, stride=100, t=FAKE, k=FAKE, p=FAKE, a=FAKE, random=FAKE,
             tokens=FAKE, probs=FAKE)
    a.update(kw)
    return lib.sample_tokens(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(logits=None), dict(logits=FAKE + 2), dict(type=3), dict(type=-1),
                                 dict(rows=1 << 31), dict(rows=1 << 28),
                                 dict(vocab=_native.MAX_VOCAB + 1), dict(stride=1 << 32), dict(random=None),
                                 dict(tokens=None), dict(t=FAKE + 1), dict(k=FAKE + 2), dict(p=FAKE + 3),
                                 dict(a=FAKE + 1), dict(random=FAKE + 2), dict(tokens=FAKE + 1), dict(probs=FAKE + 2),
                                 dict(logits=FAKE + 1, type=_native.BF16)])
def test_sample_refuses(lib, bad):
    assert sample_call(lib, **bad) == _native.EINVAL


def test_sample_of_no_rows(lib):
    assert sample_call(lib, rows=0, logits=None, random=None, tokens=None) == _native.OK


def table_args(**kw):
    a = dict(table=FAKE, stride=8, rows=4, width=8, lens=FAKE, refs=FAKE, pages=100, page_tokens=16)
    a.update(kw)
    return list(a.values())


def pool_struct(**kw):
    a = dict(planes=FAKE, n_planes=2, pages=100, page_bytes=64, page_stride=64)
    a.update(kw)
    return _native.PagePoolStruct(*a.values())


BAD_TABLES = [dict(table=None), dict(table=FAKE + 2), dict(lens=None), dict(lens=FAKE + 1), dict(refs=None),
              dict(refs=FAKE + 2), dict(stride=7), dict(stride=1 << 31), dict(rows=1 << 31), dict(width=1 << 31),
              dict(pages=1 << 31), dict(page_tokens=0), dict(page_tokens=1 << 31)]
BAD_POOLS = [dict(planes=None), dict(planes=FAKE + 4), dict(page_stride=63), dict(n_planes=1 << 20),
             dict(page_bytes=1 << 40, page_stride=1 << 41), dict(page_stride=1 << 40)]


@pytest.mark.parametrize("bad", BAD_TABLES)
def test_pages_refuse_bad_tables(lib, bad):
    ws, need = FAKE, 1 << 40
    t = table_args(**bad)
    assert lib.pages_fork(*t, None, None, None, FAKE, None, ws, need, None) == _native.EINVAL
    assert lib.pages_free(*t, FAKE, None, ws, need, None) == _native.EINVAL
    assert lib.pages_compact(None, *t, None, None, ws, need, None) == _native.EINVAL


@pytest.mark.parametrize("bad", BAD_POOLS + [dict(pages=99)])
def test_pages_refuse_bad_pools(lib, bad):
    ws, need = FAKE, 1 << 40
    pool = pool_struct(**bad)
    t = table_args()
    assert lib.pages_fork(*t, None, None, pool, FAKE, None, ws, need, None) == _native.EINVAL
    assert lib.pages_compact(pool, *t, None, None, ws, need, None) == _native.EINVAL
    if "pages" not in bad:
        assert lib.pages_copy(pool, FAKE, FAKE, 1, None, None) == _native.EINVAL


def test_pages_refuse_other_arguments(lib):
    ws, need = FAKE, 1 << 40
    t = table_args()
    fork = lambda *a: lib.pages_fork(*t, *a, ws, need, None)  # noqa: E731
    assert fork(FAKE + 1, None, None, FAKE, None) == _native.EINVAL
    assert fork(None, FAKE + 1, None, FAKE, None) == _native.EINVAL
    assert fork(None, None, None, None, None) == _native.EINVAL
    assert fork(None, None, None, FAKE + 2, None) == _native.EINVAL
    assert fork(None, None, None, FAKE, FAKE + 2) == _native.EINVAL
    assert lib.pages_free(*t, None, None, ws, need, None) == _native.EINVAL
    assert lib.pages_free(*t, FAKE + 2, None, ws, need, None) == _native.EINVAL
    assert lib.pages_free(*t, FAKE, FAKE + 2, ws, need, None) == _native.EINVAL
    assert lib.pages_compact(None, *t, FAKE + 2, None, ws, need, None) == _native.EINVAL
    assert lib.pages_compact(None, *t, None, FAKE + 2, ws, need, None) == _native.EINVAL
    assert lib.pages_copy(None, FAKE, FAKE, 1, None, None) == _native.EINVAL
    pool = pool_struct()
    assert lib.pages_copy(pool, None, FAKE, 1, None, None) == _native.EINVAL
    assert lib.pages_copy(pool, FAKE, None, 1, None, None) == _native.EINVAL
    assert lib.pages_copy(pool, FAKE + 2, FAKE, 1, None, None) == _native.EINVAL
    assert lib.pages_copy(pool, FAKE, FAKE, 1, FAKE + 2, None) == _native.EINVAL
    assert lib.pages_copy(pool, FAKE, FAKE, 1 << 31, None, None) == _native.EINVAL
    assert lib.pages_copy(pool, None, None, 0, None, None) == _native.OK
    assert lib.pages_copy(pool_struct(pages=0), FAKE, FAKE, 5, None, None) == _native.OK


def test_pages_workspace(lib):
    wb = lib.u32scan_workspace_bytes
    for pages, rows in ((1, 1), (100, 4), (4096, 4096), (1 << 20, 8192), ((1 << 31) - 1, 5)):
        need = wb(_native.OP_PAGES, pages + rows)
        assert need % 256 == 0 and need >= 12 * pages + 16 * rows
        t = table_args(pages=pages, rows=rows)
        small = need - 256
        assert lib.pages_fork(*t, None, None, None, FAKE, None, FAKE, small, None) == _native.EWORKSPACE
        assert lib.pages_free(*t, FAKE, None, FAKE, small, None) == _native.EWORKSPACE
        assert lib.pages_compact(None, *t, None, None, FAKE, small, None) == _native.EWORKSPACE
        assert lib.pages_free(*t, FAKE, None, None, need, None) == _native.EWORKSPACE
        assert lib.pages_free(*t, FAKE, None, FAKE + 16, need, None) == _native.EWORKSPACE


def test_calls_on_nothing(lib):
    t = table_args(table=None, rows=0, lens=None)
    assert lib.pages_fork(*t, None, None, None, None, None, None, 0, None) == _native.OK
    assert lib.pages_free(*t, None, None, None, 0, None) == _native.OK
    t = table_args(pages=0, refs=None)
    assert lib.pages_compact(None, *t, None, None, None, 0, None) == _native.OK


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    import u32_prefix_scan_gb300 as u

    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        u.sample_tokens(torch.zeros(4, 8), i)
    with pytest.raises(TypeError, match="torch.Tensor"):
        u.sample_tokens([[0.0]], i)
    with pytest.raises(ValueError, match="CUDA"):
        u.PagePool(torch.zeros(4, 8))
    with pytest.raises(ValueError, match="at least one plane"):
        u.PagePool([])
    with pytest.raises(ValueError, match="CUDA"):
        u.pages_free(torch.zeros(4, 8, dtype=torch.int32), i, i, 16, i)


def test_struct_matches_the_header(tmp_path):
    """The ctypes struct has the C struct's size and offsets."""
    import pathlib
    import subprocess

    root = pathlib.Path(__file__).resolve().parents[1]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "u32scan.h"\n#define O(f) offsetof('
                   'u32scan_page_pool, f)\nint main(void){printf("%zu %zu %zu %zu %zu %zu", sizeof('
                   'u32scan_page_pool), O(planes), O(n_planes), O(pages), O(page_bytes), O(page_stride));}\n')
    subprocess.check_call(["gcc", f"-I{root / 'include'}", str(src), "-o", str(tmp_path / "s")])
    got = [int(v) for v in subprocess.check_output([str(tmp_path / "s")]).split()]
    s = _native.PagePoolStruct
    assert got == [ctypes.sizeof(s), s.planes.offset, s.n_planes.offset, s.pages.offset, s.page_bytes.offset,
                   s.page_stride.offset]
