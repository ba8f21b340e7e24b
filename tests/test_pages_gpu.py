"""GPU parity of the paged cache's operations against the CPU oracle: copies
of every size and alignment, forks with and without growth until pages run
out, releases, packing; refused rows, page numbers outside the pool,
strided tables, other streams, graphs and a shared workspace."""

import numpy as np
import pytest

import oracle
from test_decode_pins import check_cache, make_cache

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def u():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from u32_prefix_scan_gb300 import build

    build.build()
    import u32_prefix_scan_gb300 as u

    return u


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().numpy()


def random_pool(seed, planes, pages, page_bytes):
    return np.random.default_rng(seed).integers(0, 256, (planes, pages, page_bytes), dtype=np.uint8)


@pytest.mark.parametrize("page_bytes", [1, 3, 4, 12, 16, 40, 48, 1000, 4096, 16384, 16400, 65537, 100000])
@pytest.mark.parametrize("planes", [1, 3])
def test_copy_sizes(u, planes, page_bytes):
    pages = 23
    pool = random_pool(page_bytes, planes, pages, page_bytes)
    perm = np.random.default_rng(1).permutation(pages).astype(np.int32)
    src, dst = perm[:9], perm[9:18]
    t = dev(pool)
    u.pages_copy(u.PagePool(t, planes_first=True), dev(src), dev(dst))
    assert np.array_equal(host(t), oracle.pages_copy(pool, src, dst))


@pytest.mark.parametrize("shift", [0, 1, 2, 4, 8, 16])
@pytest.mark.parametrize("gap", [0, 1, 4, 16])
def test_copy_alignment(u, shift, gap):
    """Planes that start anywhere, pages with gaps between them; the gaps stay."""
    pages, page_bytes = 11, 4112
    stride = page_bytes + gap
    flat = random_pool(2, 1, 1, shift + pages * stride + 16)[0, 0]
    t = dev(flat)
    plane = torch.as_strided(t, (pages, page_bytes), (stride, 1), shift)
    src, dst = np.array([0, 3, 10], np.int32), np.array([4, 5, 6], np.int32)
    u.pages_copy(u.PagePool([plane]), dev(src), dev(dst))
    for s, d in zip(src, dst):
        flat[shift + d * stride :][:page_bytes] = flat[shift + s * stride :][:page_bytes].copy()
    assert np.array_equal(host(t), flat)


def test_copy_skips_and_count(u):
    pages = 8
    pool = random_pool(3, 2, pages, 256)
    src = np.array([-1, 0, 8, 1, 2, 7, -2147483648], np.int32)
    dst = np.array([3, -1, 4, 1, 5, 6, 2], np.int32)
    t = dev(pool)
    u.pages_copy(u.PagePool(list(t.unbind(0))), dev(src), dev(dst))
    assert np.array_equal(host(t), oracle.pages_copy(pool, src, dst))
    for count in (-3, 0, 5, 6, 100):
        t = dev(pool)
        u.pages_copy(u.PagePool(t, planes_first=True), dev(src), dev(dst), dev(np.array([count], np.int32)))
        m = min(max(count, 0), 7)
        assert np.array_equal(host(t), oracle.pages_copy(pool, src[:m], dst[:m]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32, torch.int8])
def test_copy_types(u, dtype):
    layers = [torch.randn(9, 16, 2, 8, device="cuda").to(dtype) for _ in range(4)]
    was = [t.clone() for t in layers]
    u.pages_copy(u.PagePool(layers), dev(np.array([1, 2], np.int32)), dev(np.array([8, 0], np.int32)))
    for t, w in zip(layers, was):
        w[8], w[0] = w[1], w[2]
        assert torch.equal(t, w)


def run_fork(u, table, lens, refs, page_tokens, parent, grow, pool, **kw):
    t, l, r = dev(table), dev(lens), dev(refs)
    p = None if pool is None else dev(pool)
    status, left = u.pages_fork(t, l, r, page_tokens, parent=None if parent is None else dev(parent),
                                grow=None if grow is None else dev(grow),
                                pool=None if p is None else u.PagePool(p, planes_first=True), **kw)
    return host(t), host(l), host(r), host(status), int(left.item()), None if p is None else host(p)


def check_fork(u, *args):
    got, want = run_fork(u, *args), oracle.pages_fork(*args)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    return got


FORK_SHAPES = [(1, 1, 1, 4), (2, 1, 3, 1), (5, 3, 9, 7), (40, 7, 120, 16), (300, 30, 4000, 16), (257, 40, 9000, 3),
               (1500, 6, 5000, 32)]


@pytest.mark.parametrize("rows,width,pages,page_tokens", FORK_SHAPES)
@pytest.mark.parametrize("what", ["grow", "fork", "both", "wild"])
def test_fork(u, rows, width, pages, page_tokens, what):
    rng = np.random.default_rng(rows + width)
    active = rows - rows // 3 if what != "grow" else rows
    table, lens, refs = make_cache(rows, rows, width, pages, page_tokens, empty_from=active)
    parent, grow = np.full(rows, -1, np.int32), np.zeros(rows, np.int32)
    if what != "grow":
        parent[active:] = rng.integers(0, active, rows - active)
    if what != "fork":
        grow[:] = rng.choice([0, 1, 1, 2, 5 * page_tokens], rows)
    if what == "wild":  # arguments to refuse, among good ones
        bad = rng.random(rows) < 0.2
        parent[bad] = rng.integers(-5, rows + 5, bad.sum())
        grow[rng.random(rows) < 0.1] = -1
        grow[rng.random(rows) < 0.1] = 2**31 - 1
    pool = random_pool(1, 2, pages, 48)
    args = (table, lens, refs, page_tokens, parent if what != "grow" else None, grow if what != "fork" else None, pool)
    t, l, r, status, left, _ = check_fork(u, *args)
    check_cache(t, l, r, page_tokens)
    assert left == (r == 0).sum()


@pytest.mark.parametrize("pages", [1, 4095, 4096, 4097, 100003, 1 << 20])
@pytest.mark.parametrize("need", [1, 100, 5000])
def test_fork_takes_the_lowest_free_pages(u, pages, need):
    """Growth alone, free pages scattered over many tiles, enough or not."""
    rng = np.random.default_rng(pages)
    refs = (rng.random(pages) < 0.97).astype(np.int32)
    rows = 8
    table = np.full((rows, need), -1, np.int32)
    lens = np.zeros(rows, np.int32)
    grow = np.full(rows, need, np.int32)
    check_fork(u, table, lens, refs, 1, None, grow, None)


def test_fork_no_free_and_all_free(u):
    table, lens = np.full((3, 4), -1, np.int32), np.zeros(3, np.int32)
    for refs in (np.ones(5000, np.int32), np.zeros(5000, np.int32)):
        check_fork(u, table, lens, refs, 8, None, np.array([9, 0, 32], np.int32), None)
    check_fork(u, table, lens, np.zeros(0, np.int32), 8, None, np.array([9, 0, 32], np.int32), None)
    check_fork(u, np.zeros((0, 4), np.int32), np.zeros(0, np.int32), np.zeros(70, np.int32), 8, None, None, None)
    check_fork(u, np.zeros((3, 0), np.int32), lens, np.zeros(70, np.int32), 8, np.array([-1, 0, -1], np.int32),
               np.array([0, 0, 1], np.int32), None)


@pytest.mark.parametrize("rows", [65535, 65536, 70001])
@pytest.mark.parametrize("pages", [3000, 300000])
def test_fork_many_rows(u, rows, pages):
    """More rows than one packed scan takes; pages for some and for all."""
    rng = np.random.default_rng(rows)
    table = np.full((rows, 3), -1, np.int32)
    lens, refs = np.zeros(rows, np.int32), np.zeros(pages, np.int32)
    active = 1000
    lens[:active] = rng.integers(0, 9, active)
    n = -(-lens // 4)
    place = rng.permutation(pages)
    for j in range(3):
        hold = np.flatnonzero(n > j)
        table[hold, j], place = place[: hold.size], place[hold.size :]
    refs[table[table >= 0]] = 1
    parent = np.full(rows, -1, np.int32)
    parent[active:] = np.where(rng.random(rows - active) < 0.5, rng.integers(0, active, rows - active), -1)
    check_fork(u, table, lens, refs, 4, parent, rng.integers(0, 5, rows).astype(np.int32), random_pool(3, 1, pages, 16))


def test_fork_long_rows(u):
    """A prefix of many table chunks shared by many children."""
    rows, width, pages, page_tokens = 40, 3001, 8000, 2
    table, lens, refs = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32), np.zeros(pages, np.int32)
    table[3, :2777] = np.random.default_rng(0).permutation(pages)[:2777]
    lens[3] = 2777 * 2 - 1
    refs[table[3, :2777]] = 1
    parent = np.full(rows, 3, np.int32)
    parent[3] = -1
    check_fork(u, table, lens, refs, page_tokens, parent, np.ones(rows, np.int32), random_pool(0, 1, pages, 20))


def test_fork_passes_over_foreign_pages(u):
    """Entries outside the pool are copied to the child and nothing else."""
    table = np.array([[5, -1, 2**31 - 1, 70, 1], [-1] * 5], np.int32)
    lens, refs = np.array([17, 0], np.int32), np.array([0, 1, 0, 0, 0, 1, 0], np.int32)
    check_fork(u, table, lens, refs, 4, np.array([-1, 0], np.int32), None, random_pool(0, 1, 7, 16))


def run_free(u, table, lens, refs, page_tokens, release):
    t, l, r = dev(table), dev(lens), dev(refs)
    freed = u.pages_free(t, l, r, page_tokens, dev(release))
    return host(t), host(l), host(r), int(freed.item())


@pytest.mark.parametrize("rows,width,pages,page_tokens", FORK_SHAPES + [(9000, 4, 20000, 1), (3, 5000, 9000, 2)])
@pytest.mark.parametrize("share", [0.0, 0.4, 1.0])
def test_free(u, rows, width, pages, page_tokens, share):
    table, lens, refs = make_cache(rows, rows, width, pages, page_tokens)
    release = (np.random.default_rng(1).random(rows) < share) * np.random.default_rng(2).integers(-9, -1, rows)
    args = (table, lens, refs, page_tokens, release.astype(np.int32))
    got, want = run_free(u, *args), oracle.pages_free(*args)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    check_cache(got[0], got[1], got[2], page_tokens)


def test_free_odd_rows(u):
    table = np.array([[1, -1, 9, 2], [3, 3, 0, 0], [0, 1, 2, 3], [2, 2, 2, 2]], np.int32)
    lens = np.array([14, -5, 2**31 - 1, 0], np.int32)  # foreign pages, a negative and an impossible length
    refs = np.array([2, 2, 2, 2], np.int32)
    args = (table, lens, refs, 4, np.ones(4, np.int32))
    for g, w in zip(run_free(u, *args), oracle.pages_free(*args)):
        assert np.array_equal(g, w)
    args = (np.zeros((0, 4), np.int32), np.zeros(0, np.int32), refs, 4, np.zeros(0, np.int32))
    assert run_free(u, *args)[3] == 0


def run_compact(u, table, lens, refs, page_tokens, pool):
    t, l, r = dev(table), dev(lens), dev(refs)
    p = None if pool is None else dev(pool)
    live, remap = u.pages_compact(None if p is None else u.PagePool(p, planes_first=True), t, l, r, page_tokens)
    assert np.array_equal(host(l), lens)
    return host(t), host(r), int(live.item()), host(remap), None if p is None else host(p)


def check_compact(u, *args):
    got, want = run_compact(u, *args), oracle.pages_compact(*args)
    for g, w in zip(got[:4], want[:4]):
        assert np.array_equal(g, w)
    if args[4] is not None:
        # bytes of pages that are free afterwards are the mover's old ones in both
        assert np.array_equal(got[4], want[4])
    return got


@pytest.mark.parametrize("rows,width,pages,page_tokens", FORK_SHAPES + [(600, 20, 4096, 4), (700, 30, 20011, 4)])
@pytest.mark.parametrize("page_bytes", [0, 48, 20000])
def test_compact(u, rows, width, pages, page_tokens, page_bytes):
    if pages * page_bytes > 1 << 27:
        pytest.skip("large pages are tested on the small caches")
    table, lens, refs = make_cache(rows, rows, width, pages, page_tokens)
    pool = random_pool(1, 2, pages, page_bytes) if page_bytes else None
    t, r, live, remap, _ = check_compact(u, table, lens, refs, page_tokens, pool)
    check_cache(t, lens, r, page_tokens)
    assert np.all(r[:live] != 0) and np.all(r[live:] == 0)


@pytest.mark.parametrize("pages", [1, 2, 31, 4096, 8192, 8193, 50000])
@pytest.mark.parametrize("kind", ["none", "all", "front", "back", "half", "one_high"])
def test_compact_patterns(u, pages, kind):
    """refs alone, at tile boundaries: nothing to move, all to move."""
    refs = np.zeros(pages, np.int32)
    if kind == "all":
        refs[:] = 3
    elif kind == "front":
        refs[: pages // 2] = 1
    elif kind == "back":
        refs[pages - pages // 2 :] = np.arange(pages // 2) + 1
    elif kind == "half":
        refs[::2] = np.arange(pages)[::2] + 1
    elif kind == "one_high":
        refs[-1] = 7
    table, lens = np.full((1, 1), -1, np.int32), np.zeros(1, np.int32)
    check_compact(u, table, lens, refs, 1, random_pool(2, 1, pages, 8))


def test_compact_leaves_foreign_entries(u):
    table = np.array([[7, -1, 99, 6, 2**31 - 1, 0]], np.int32)
    refs = np.array([1, 0, 0, 0, 0, 0, 0, 1], np.int32)  # entry 6 is in use but its page is free
    check_compact(u, table, np.array([6], np.int32), refs, 1, random_pool(2, 1, 8, 64))


def test_strided_tables(u):
    rows, width, pages = 50, 9, 400
    table, lens, refs = make_cache(3, rows, width, pages, 4, empty_from=30)
    parent = np.full(rows, -1, np.int32)
    parent[30:] = np.arange(20)
    wide = np.full((rows, width + 5), 7777, np.int32)
    wide[:, 2 : 2 + width] = table
    w, l, r = dev(wide), dev(lens), dev(refs)
    view = w[:, 2 : 2 + width]
    u.pages_fork(view, l, r, 4, parent=dev(parent))
    release = np.arange(rows, dtype=np.int32) % 3
    u.pages_free(view, l, r, 4, dev(release))
    u.pages_compact(None, view, l, r, 4)
    t2, l2, r2, _, _, _ = oracle.pages_fork(table, lens, refs, 4, parent)
    t2, l2, r2, _ = oracle.pages_free(t2, l2, r2, 4, release)
    t2, r2, _, _, _ = oracle.pages_compact(t2, l2, r2, 4)
    got = host(w)
    assert np.array_equal(got[:, 2 : 2 + width], t2)
    assert np.all(got[:, :2] == 7777) and np.all(got[:, 2 + width :] == 7777)
    assert np.array_equal(host(l), l2) and np.array_equal(host(r), r2)


def test_workspace_shared_with_the_scans(u):
    """Page operations between scans, sorts and folds on one workspace."""
    from u32_prefix_scan_gb300 import inputs

    rows, width, pages = 100, 12, 9000
    table, lens, refs = make_cache(4, rows, width, pages, 4, empty_from=60)
    parent = np.full(rows, -1, np.int32)
    parent[60:] = np.arange(40)
    a = inputs.splitmix_u32(5, 0, 300007)
    keys = inputs.splitmix_u32(6, 0, 20001)
    for _ in range(3):
        for step in range(3):
            d = dev(a.view(np.int32).copy())
            u.scan_exclusive_u32(d)
            assert np.array_equal(host(d).view(np.uint32), oracle.scan_exclusive(a)[0])
            perm = u.radix_sort_perm_u32(dev(keys.view(np.int32)))
            assert np.array_equal(host(perm), oracle.sort_perm(keys))
            assert int(u.reduce_u32_op(dev(a.view(np.int32)), "max").item()) & 0xFFFFFFFF == int(a.max())
            if step == 0:
                check_fork(u, table, lens, refs, 4, parent, None, None)
            elif step == 1:
                args = (table, lens, refs, 4, np.ones(rows, np.int32))
                for g, w in zip(run_free(u, *args), oracle.pages_free(*args)):
                    assert np.array_equal(g, w)
            else:
                check_compact(u, table, lens, refs, 4, None)
    u.check()


def test_other_stream_and_graph(u):
    rows, width, pages = 64, 12, 1000
    table, lens, refs = make_cache(8, rows, width, pages, 4, empty_from=40)
    parent = np.full(rows, -1, np.int32)
    parent[40:] = np.arange(24)
    grow = np.ones(rows, np.int32)
    pool = random_pool(5, 2, pages, 64)
    release = (np.arange(rows) % 2).astype(np.int32)
    t2, l2, r2, s2, left2, p2 = oracle.pages_fork(table, lens, refs, 4, parent, grow, pool)
    t2, l2, r2, f2 = oracle.pages_free(t2, l2, r2, 4, release)
    t2, r2, n2, m2, p2 = oracle.pages_compact(t2, l2, r2, 4, p2)
    start = [dev(x) for x in (table, lens, refs, pool)]
    t, l, r, p = work = [x.clone() for x in start]
    handle = u.PagePool(p, planes_first=True)
    par, g, rel = dev(parent), dev(grow), dev(release)
    status = torch.empty(rows, dtype=torch.int32, device="cuda")
    left, freed, live = (torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(3))
    remap = torch.empty(pages, dtype=torch.int32, device="cuda")
    ws = u.Workspace(u._native.lib().u32scan_workspace_bytes(9, pages + rows), t.device)

    def step(stream):
        kw = dict(stream=stream, workspace=ws)
        u.pages_fork(t, l, r, 4, parent=par, grow=g, pool=handle, status=status, free_pages=left, **kw)
        u.pages_free(t, l, r, 4, rel, freed=freed, **kw)
        u.pages_compact(handle, t, l, r, 4, live=live, remap=remap, **kw)

    def verify():
        torch.cuda.synchronize()
        for got, want in zip((t, l, r, p, status, remap), (t2, l2, r2, p2, s2, m2)):
            assert np.array_equal(host(got), want)
        assert [int(x.item()) for x in (left, freed, live)] == [left2, f2, n2]

    torch.cuda.synchronize()
    step(torch.cuda.Stream())
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, s in zip(work, start):
            x.copy_(s)
        step(None)
    for _ in range(3):
        graph.replay()
        verify()


def test_refusals(u):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, refs = i32(4, 8), i32(4), i32(50)
    with pytest.raises(TypeError, match="table"):
        u.pages_free(table.long(), lens, refs, 4, lens)
    with pytest.raises(ValueError, match="two dimensions"):
        u.pages_free(table[0], lens, refs, 4, lens)
    with pytest.raises(ValueError, match="adjacent"):
        u.pages_free(i32(8, 4).t(), lens, refs, 4, lens)
    with pytest.raises(ValueError, match="overlap"):
        u.pages_free(i32(1, 8).expand(4, 8), lens, refs, 4, lens)
    with pytest.raises(ValueError, match="lens"):
        u.pages_free(table, i32(3), refs, 4, lens)
    with pytest.raises(ValueError, match="at least 4"):
        u.pages_free(table, lens, refs, 4, i32(3))
    with pytest.raises(u._native.U32ScanError):
        u.pages_free(table, lens, refs, 0, lens)
    with pytest.raises(TypeError, match="PagePool"):
        u.pages_compact(table, table, lens, refs, 4)
    with pytest.raises(ValueError, match="at least 50"):
        u.pages_compact(None, table, lens, refs, 4, remap=i32(49))
    with pytest.raises(u._native.U32ScanError):  # a pool of another size
        u.pages_compact(u.PagePool(i32(49, 8)), table, lens, refs, 4)
    with pytest.raises(ValueError, match="agree"):
        u.PagePool([i32(4, 8), i32(4, 9)])
    with pytest.raises(ValueError, match="adjacent"):
        u.PagePool(i32(4, 8, 8).transpose(1, 2))
    with pytest.raises(ValueError, match="overlap"):
        u.PagePool(i32(1, 8).expand(4, 8))
    with pytest.raises(ValueError, match="differ"):
        u.pages_copy(u.PagePool(i32(4, 8)), i32(2), i32(3))
