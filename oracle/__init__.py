"""CPU oracle for the U32 scan primitives (numpy front end over oracle.c).

TEST INFRASTRUCTURE. Only the tests, the smoke check and the benchmark's
CPU-baseline / reference legs may import this package. The CUDA library and
its Python binding never import it, and it imports nothing from them: the two
share no code. Inputs come from the seeded generator module, passed in as
arrays.

Every wrapper copies its inputs, calls one plain sequential C function
(oracle.c, one thread) and returns new arrays; see oracle.c for the passage
of the source pages each function follows. Nothing here is tuned.

Parity pins: every function is pinned in tests/test_oracle_pins.py against
values the pages print (tests/golden/), closed forms, invariants the pages
state, independent library routines (numpy) and brute force on tiny inputs.
"""

from __future__ import annotations

import ctypes
import os
import pathlib
import subprocess

import numpy as np

_HERE = pathlib.Path(__file__).resolve().parent
_SRC = _HERE / "oracle.c"
_SO = _HERE / "liboracle.so"

_u32p = ctypes.POINTER(ctypes.c_uint32)
_i32p = ctypes.POINTER(ctypes.c_int32)
_u64 = ctypes.c_uint64

_lib = None


def build(force: bool = False) -> pathlib.Path:
    """Compile oracle.c into liboracle.so (plain gcc -O2, no target flags)."""
    if force or not _SO.exists() or _SO.stat().st_mtime < _SRC.stat().st_mtime:
        tmp = _SO.with_suffix(f".so.tmp{os.getpid()}")
        subprocess.check_call(
            ["gcc", "-O2", "-std=c11", "-Wall", "-Wextra", "-shared", "-fPIC",
             "-o", str(tmp), str(_SRC), "-lm"])
        os.replace(tmp, _SO)
    return _SO


def _configure(lib):
    """Declare the C signatures on a loaded oracle library."""
    f32, i32, u8p = ctypes.c_float, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint8)
    table = [_i32p, _u64, _u64, _i32p, _i32p, _u64, _u64]  # table, rows, width, lens, refs, pages, page_tokens
    lib.oracle_sample_token.argtypes = [ctypes.POINTER(f32), _u64, f32, i32, f32, f32, ctypes.c_uint32,
                                        ctypes.POINTER(f32)]
    lib.oracle_sample_token.restype = i32
    lib.oracle_pages_copy.argtypes = [u8p, _u64, _u64, _u64, _i32p, _i32p, _u64]
    lib.oracle_pages_copy.restype = None
    lib.oracle_pages_fork.argtypes = [*table, _i32p, _i32p, u8p, _u64, _u64, _i32p]
    lib.oracle_pages_fork.restype = i32
    lib.oracle_pages_free.argtypes = [*table, _i32p]
    lib.oracle_pages_free.restype = i32
    lib.oracle_pages_compact.argtypes = [*table, u8p, _u64, _u64, _i32p]
    lib.oracle_pages_compact.restype = i32
    f32p, f64p = ctypes.POINTER(f32), ctypes.POINTER(ctypes.c_double)
    lib.oracle_adjust_row.argtypes = [f32p, _u64, _i32p, ctypes.c_int64, ctypes.c_int64, f32, f32, f32, _i32p, f32p,
                                      _u64, _u32p, f32p, u8p]
    lib.oracle_adjust_row.restype = None
    lib.oracle_code_value.argtypes = [ctypes.c_uint8]
    lib.oracle_code_value.restype = f32
    lib.oracle_value_code.argtypes = [f32]
    lib.oracle_value_code.restype = ctypes.c_uint8
    lib.oracle_rotate_head.argtypes = [f32p, _u64, f32p, f32p, _u64, ctypes.c_int, f32p]
    lib.oracle_rotate_head.restype = None
    lib.oracle_append_block.argtypes = [f32p, _u64, _u64, _u64, u8p, _u64, f32]
    lib.oracle_append_block.restype = f32
    lib.oracle_attend_query.argtypes = [f64p, f64p, f64p, u8p, _u64, _u64, ctypes.c_double, f64p]
    lib.oracle_attend_query.restype = None
    lib.oracle_scan_exclusive_u32.argtypes = [_u32p, _u64]
    lib.oracle_scan_exclusive_u32.restype = ctypes.c_uint32
    lib.oracle_scan_inclusive_u32.argtypes = [_u32p, _u64]
    lib.oracle_scan_inclusive_u32.restype = ctypes.c_uint32
    lib.oracle_scan_op_u32.argtypes = [ctypes.c_int, ctypes.c_int, _u32p, _u64]
    lib.oracle_scan_op_u32.restype = ctypes.c_uint32
    lib.oracle_scan_blocked_u32.argtypes = [ctypes.c_int, ctypes.c_uint, _u32p, _u64, _u32p]
    lib.oracle_scan_blocked_u32.restype = ctypes.c_uint32
    lib.oracle_segscan_inclusive_u32.argtypes = [_u32p, _i32p, _u64]
    lib.oracle_segscan_inclusive_u32.restype = None
    lib.oracle_segreduce_u32.argtypes = [_u32p, _i32p, _u64, _u32p]
    lib.oracle_segreduce_u32.restype = ctypes.c_uint64
    lib.oracle_compact_indices.argtypes = [_i32p, _u64, _i32p, _i32p, _i32p]
    lib.oracle_compact_indices.restype = ctypes.c_int32
    lib.oracle_radix_perm_bits.argtypes = [_u32p, _u64, ctypes.c_uint, _i32p, _i32p, _i32p]
    lib.oracle_radix_perm_bits.restype = None
    lib.oracle_sort_perm_u32.argtypes = [_u32p, _u64, _i32p]
    lib.oracle_sort_perm_u32.restype = ctypes.c_int
    lib.oracle_runs_layout_u32.argtypes = [_u32p, _u64, _u32p]
    lib.oracle_runs_layout_u32.restype = ctypes.c_uint32
    lib.oracle_runs_fill_owner.argtypes = [_u32p, _u32p, _u64, _i32p, _u64]
    lib.oracle_runs_fill_owner.restype = None
    lib.oracle_compact_values_u32.argtypes = [_u32p, _i32p, _u64, _u32p]
    lib.oracle_compact_values_u32.restype = ctypes.c_uint64
    lib.oracle_scan_op_u64.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_uint64), _u64]
    lib.oracle_scan_op_u64.restype = ctypes.c_uint64
    return lib


def _load():
    global _lib
    if _lib is None:
        _lib = _configure(ctypes.CDLL(str(build())))
    return _lib


def _u32(a) -> np.ndarray:
    a = np.asarray(a)
    if a.dtype != np.uint32:
        if a.size and (a.min() < 0 or a.max() >= (1 << 32)):
            raise ValueError("values must lie in [0, 2^32)")
        a = a.astype(np.uint32)
    return np.ascontiguousarray(a).copy()


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32)).copy()


def _p(a: np.ndarray, t):
    return a.ctypes.data_as(t)


def scan_exclusive(a):
    """(scanned copy, total): out[j] = a[0] + .. + a[j-1] mod 2^32."""
    out = _u32(a)
    total = _load().oracle_scan_exclusive_u32(_p(out, _u32p), out.size)
    return out, int(total)


def scan_inclusive(a):
    """(scanned copy, total): out[j] = a[0] + .. + a[j] mod 2^32."""
    out = _u32(a)
    total = _load().oracle_scan_inclusive_u32(_p(out, _u32p), out.size)
    return out, int(total)


SCAN_OPS = {"add": 0, "mul": 1, "and": 2, "or": 3, "xor": 4, "min": 5, "max": 6}


def scan_op(a, op: str, inclusive: bool):
    """(scanned copy, fold) under one of the CAIRN integer operators on
    uint32: add, mul (both wrapping), and, or, xor, min, max."""
    out = _u32(a)
    total = _load().oracle_scan_op_u32(SCAN_OPS[op], int(bool(inclusive)), _p(out, _u32p), out.size)
    return out, int(total)


def scan_blocked(a, b: int, inclusive: bool):
    """The three-pass blocked scan at fork depth b: (scanned copy, total)."""
    out = _u32(a)
    d = min(int(b), 30, max(out.size, 1).bit_length() - 1)
    scratch = np.zeros(1 << d, dtype=np.uint32)
    total = _load().oracle_scan_blocked_u32(int(bool(inclusive)), int(b), _p(out, _u32p),
                                            out.size, _p(scratch, _u32p))
    return out, int(total)


def segscan_inclusive(a, flags):
    """Segmented inclusive scan (copy); a non-zero flag opens a segment."""
    out = _u32(a)
    f = _i32(flags)
    if f.size != out.size:
        raise ValueError("values and flags differ in length")
    _load().oracle_segscan_inclusive_u32(_p(out, _u32p), _p(f, _i32p), out.size)
    return out


def segreduce(a, flags):
    """(per-segment wrapped sums in segment order, number of segments)."""
    v = _u32(a)
    f = _i32(flags)
    if f.size != v.size:
        raise ValueError("values and flags differ in length")
    sums = np.zeros(max(v.size, 1), dtype=np.uint32)
    nseg = _load().oracle_segreduce_u32(_p(v, _u32p), _p(f, _i32p), v.size, _p(sums, _u32p))
    return sums[:nseg].copy(), int(nseg)


def compact_indices(flags):
    """(inclusive offsets, indices with a -1 tail, count)."""
    f = _i32(flags)
    n = f.size
    if n >= (1 << 31):
        raise ValueError("n must be below 2^31")
    offsets = np.empty(n, dtype=np.int32)
    indices = np.empty(n, dtype=np.int32)
    count = np.zeros(1, dtype=np.int32)
    _load().oracle_compact_indices(_p(f, _i32p), n, _p(offsets, _i32p), _p(indices, _i32p),
                                   _p(count, _i32p))
    return offsets, indices, int(count[0])


def radix_perm_bits(keys, bits: int = 32):
    """The sort graph's permutation: LSD, one bit per pass, `bits` passes."""
    k = _u32(keys)
    n = k.size
    if n >= (1 << 31):
        raise ValueError("n must be below 2^31")
    if not 1 <= bits <= 32:
        raise ValueError("bits must be in 1..32")
    perm = np.empty(n, dtype=np.int32)
    zeros = np.empty(n, dtype=np.int32)
    slots = np.empty(n, dtype=np.int32)
    _load().oracle_radix_perm_bits(_p(k, _u32p), n, bits, _p(perm, _i32p), _p(zeros, _i32p),
                                   _p(slots, _i32p))
    return perm


def sort_perm(keys):
    """The unique stable sorting permutation, by (key, index) order."""
    k = _u32(keys)
    n = k.size
    if n >= (1 << 31):
        raise ValueError("n must be below 2^31")
    perm = np.empty(n, dtype=np.int32)
    if _load().oracle_sort_perm_u32(_p(k, _u32p), n, _p(perm, _i32p)) != 0:
        raise MemoryError("oracle_sort_perm_u32 could not allocate")
    return perm


def runs_layout(counts):
    """(ends, entries): ends the inclusive scan of the counts (mod 2^32),
    entries = max(total, 1)."""
    c = _u32(counts)
    ends = np.empty(c.size, dtype=np.uint32)
    entries = _load().oracle_runs_layout_u32(_p(c, _u32p), c.size, _p(ends, _u32p))
    return ends, int(entries)


def runs_owner(counts):
    """(ends, entries, owner row): the runs layout, then its `entries` slots
    filled by the scatter over the owners with each owner's index, so that
    slot e holds owner(e, ends); -1 where no run reaches."""
    c = _u32(counts)
    if c.size >= (1 << 31):
        raise ValueError("n must be below 2^31")
    ends, entries = runs_layout(c)
    slots = np.empty(entries, dtype=np.int32)
    _load().oracle_runs_fill_owner(_p(c, _u32p), _p(ends, _u32p), c.size, _p(slots, _i32p), entries)
    return ends, entries, slots


def compact_values(values, flags=None, out=None):
    """(out, count): the kept values in order at the front of a copy of
    `out` (zeros when not given), the rest of it unchanged. An element is
    kept when its flag is non-zero, or, with no flags, its value is."""
    v = _u32(values)
    o = np.zeros(v.size, dtype=np.uint32) if out is None else _u32(out)
    if o.size != v.size:
        raise ValueError("out must have n elements")
    f = None if flags is None else _i32(flags)
    if f is not None and f.size != v.size:
        raise ValueError("values and flags differ in length")
    used = _load().oracle_compact_values_u32(_p(v, _u32p), None if f is None else _p(f, _i32p), v.size,
                                            _p(o, _u32p))
    return o, int(used)


def scan_op_u64(a, op: str, inclusive: bool):
    """(scanned copy, fold) of a uint64 row under one of the CAIRN integer
    operators (add and mul wrap at 2^64)."""
    out = np.ascontiguousarray(np.asarray(a, dtype=np.uint64)).copy()
    total = _load().oracle_scan_op_u64(SCAN_OPS[op], int(bool(inclusive)),
                                       out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), out.size)
    return out, int(total)


def sample_tokens(logits, random, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens, probs) of float32 logits [rows, vocab] under per-row
    temperature, top_k, top_p and min_p (None: 1 and no filter), drawn with
    the uint32 words `random`."""
    x = np.ascontiguousarray(np.asarray(logits, dtype=np.float32))
    rows, n = x.shape
    words = np.asarray(random).astype(np.uint32)

    def values(v, none):
        return np.full(rows, none) if v is None else np.asarray(v)

    t, k, p, a = values(temperature, 1.0), values(top_k, 0), values(top_p, 1.0), values(min_p, 0.0)
    tokens, probs = np.empty(rows, dtype=np.int32), np.empty(rows, dtype=np.float32)
    prob = ctypes.c_float()
    for b in range(rows):
        row = np.ascontiguousarray(x[b])
        tokens[b] = _load().oracle_sample_token(row.ctypes.data_as(ctypes.POINTER(ctypes.c_float)), n, float(t[b]),
                                                int(k[b]), float(p[b]), float(a[b]), int(words[b]),
                                                ctypes.byref(prob))
        probs[b] = prob.value
    return tokens, probs


def _cache(table, lens, refs):
    return _i32(table).copy(), _i32(lens).copy(), _i32(refs).copy()


def _bytes(pool, pages):
    """(copy as [planes, pages, page_bytes] bytes, pointer, planes, page_bytes) of a pool, or of none."""
    if pool is None:
        return None, None, 0, 0
    p = np.ascontiguousarray(np.asarray(pool, dtype=np.uint8)).copy()
    if p.ndim != 3 or p.shape[1] != pages:
        raise ValueError("pool must be [planes, pages, page_bytes]")
    return p, p.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8)), p.shape[0], p.shape[2]


def pages_copy(pool, src, dst):
    """The pool [planes, pages, page_bytes] after copying page src[i] to dst[i]."""
    p, ptr, planes, page_bytes = _bytes(pool, np.asarray(pool).shape[1])
    s, d = _i32(src), _i32(dst)
    _load().oracle_pages_copy(ptr, planes, p.shape[1], page_bytes, _p(s, _i32p), _p(d, _i32p), s.size)
    return p


def pages_fork(table, lens, refs, page_tokens, parent=None, grow=None, pool=None):
    """(table, lens, refs, status, free pages left, pool) after the fork."""
    t, l, r = _cache(table, lens, refs)
    p, ptr, planes, page_bytes = _bytes(pool, r.size)
    par = None if parent is None else _i32(parent)
    g = None if grow is None else _i32(grow)
    status = np.empty(l.size, dtype=np.int32)
    left = _load().oracle_pages_fork(_p(t, _i32p), t.shape[0], t.shape[1], _p(l, _i32p), _p(r, _i32p), r.size,
                                     page_tokens, None if par is None else _p(par, _i32p),
                                     None if g is None else _p(g, _i32p), ptr, planes, page_bytes, _p(status, _i32p))
    return t, l, r, status, int(left), p


def pages_free(table, lens, refs, page_tokens, release):
    """(table, lens, refs, pages that became free) after the release."""
    t, l, r = _cache(table, lens, refs)
    rel = _i32(release)
    freed = _load().oracle_pages_free(_p(t, _i32p), t.shape[0], t.shape[1], _p(l, _i32p), _p(r, _i32p), r.size,
                                      page_tokens, _p(rel, _i32p))
    return t, l, r, int(freed)


def pages_compact(table, lens, refs, page_tokens, pool=None):
    """(table, refs, live, remap, pool) after packing the live pages."""
    t, l, r = _cache(table, lens, refs)
    p, ptr, planes, page_bytes = _bytes(pool, r.size)
    remap = np.empty(r.size, dtype=np.int32)
    live = _load().oracle_pages_compact(_p(t, _i32p), t.shape[0], t.shape[1], _p(l, _i32p), _p(r, _i32p), r.size,
                                        page_tokens, ptr, planes, page_bytes, _p(remap, _i32p))
    return t, r, int(live), remap, p


def _f32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.float32))


def _fp(a):
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_float))


def _up(a):
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8))


def adjust_logits(logits, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None,
                  frequency=None, bias_tokens=None, bias=None, allowed=None):
    """(adjusted, touched): float32 logits [rows, vocab] under a request's
    rules, before they are rounded to their type, and which of them a rule
    reached."""
    x = _f32(logits)
    rows, vocab = x.shape
    h = np.zeros((rows, 0), np.int32) if history is None else _i32(history)
    held = np.full(rows, h.shape[1]) if history_lens is None else np.clip(history_lens, 0, h.shape[1])
    prompt = np.zeros(rows, np.int64) if prompt_lens is None else np.clip(prompt_lens, 0, held)
    none = np.full(rows, np.nan, np.float32)
    r, p, f = (none if v is None else _f32(v) for v in (repetition, presence, frequency))
    names = np.zeros((rows, 0), np.int32) if bias_tokens is None else _i32(bias_tokens)
    adds = np.zeros((rows, 0), np.float32) if bias is None else _f32(bias)
    out, touched = np.empty_like(x), np.empty(x.shape, np.uint8)
    for b in range(rows):
        mask = None if allowed is None else _u32(allowed[b])
        hb, nb, ab = np.ascontiguousarray(h[b]), np.ascontiguousarray(names[b]), np.ascontiguousarray(adds[b])
        _load().oracle_adjust_row(_fp(x[b]), vocab, _p(hb, _i32p), int(held[b]), int(prompt[b]), float(r[b]),
                                  float(p[b]), float(f[b]), _p(nb, _i32p), _fp(ab), nb.size,
                                  None if mask is None else _p(mask, _u32p), _fp(out[b]), _up(touched[b]))
    return out, touched.astype(bool)


def code_values(codes):
    """float32 values of uint8 codes (8 bits: sign, 4 of exponent, 3 of fraction)."""
    table = np.array([_load().oracle_code_value(c) for c in range(256)], np.float32)
    return table[np.asarray(codes, np.uint8)]


def value_codes(x):
    """The nearest codes (uint8) of float32 values."""
    flat = _f32(x).ravel()
    return np.array([_load().oracle_value_code(float(v)) for v in flat], np.uint8).reshape(np.shape(x))


def _row_tokens(lens, starts, tokens, s):
    """(begin, n, first position) of row s's tokens."""
    if starts is None:
        return s, 1, int(lens[s]) - 1
    b, e = (min(max(int(v), 0), tokens) for v in starts[s : s + 2])
    n = max(e - b, 0)
    return b, n, int(lens[s]) - n


def rotate_heads(x, cos_row, sin_row, interleaved=False):
    """One token's heads [heads, dim] (float32) rotated."""
    x, c, s = _f32(x), _f32(cos_row), _f32(sin_row)
    out = np.empty_like(x)
    for h in range(x.shape[0]):
        _load().oracle_rotate_head(_fp(x[h]), x.shape[1], _fp(c), _fp(s), c.size, int(interleaved), _fp(out[h]))
    return out


def pages_append(keys, values, table, lens, new_keys, new_values, starts=None, status=None, cos=None, sin=None,
                 interleaved=False, key_scales=None, value_scales=None, queries=None, queries_out=None):
    """(keys, values, key_scales, value_scales, queries_out) after the append.
    keys, values: [pages, page_tokens, heads, dim], float32 (the caller
    rounds them to the cache's type) or, with scales [pages, blocks, heads],
    uint8 codes; queries_out: what it held before."""
    keys, values, table, lens = keys.copy(), values.copy(), _i32(table), _i32(lens)
    ks, vs = (None if a is None else _f32(a).copy() for a in (key_scales, value_scales))
    pages, page_tokens, heads, dim = keys.shape
    size = page_tokens // ks.shape[1] if ks is not None else page_tokens
    tokens = new_keys.shape[0]
    q = None if queries is None else _f32(queries_out).copy()
    turn = cos is not None and np.shape(cos)[1] > 0
    for s in range(lens.size):
        begin, n, first = _row_tokens(lens, starts, tokens, s)
        held, turned = [], {}
        for i in range(n):
            at = first + i
            reached = not turn or 0 <= at < len(cos)
            if q is not None:
                row = _f32(queries[begin + i])
                q[begin + i] = (rotate_heads(row, cos[at], sin[at], interleaved) if turn else row) if reached else np.nan
            if at < 0 or not reached or (status is not None and status[s] < 0) or at // page_tokens >= table.shape[1]:
                continue
            if not 0 <= table[s, at // page_tokens] < pages:
                continue
            k = _f32(new_keys[begin + i])
            turned[at] = (rotate_heads(k, cos[at], sin[at], interleaved) if turn else k, _f32(new_values[begin + i]))
            held.append(at)
        if ks is None:
            for at in held:
                p, t = table[s, at // page_tokens], at % page_tokens
                keys[p, t], values[p, t] = turned[at]
            continue
        for at in held:
            if at % size and at - 1 in turned:
                continue  # not the first new one of its block
            p, t = int(table[s, at // page_tokens]), at % page_tokens
            last = at
            while last + 1 in turned and (last + 1) % size:
                last += 1
            before, block = t % size, t // size
            for which, codes, scales in ((0, keys, ks), (1, values, vs)):
                for h in range(heads):
                    x = _f32([turned[j][which][h] for j in range(at, last + 1)])
                    part = np.ascontiguousarray(codes[p, t - before : t - before + size, h])
                    scales[p, block, h] = _load().oracle_append_block(_fp(x), len(x), dim, before, _up(part), dim,
                                                                      float(scales[p, block, h]))
                    codes[p, t - before : t - before + size, h] = part
    return keys, values, ks, vs, q


def pages_attend(queries, keys, values, key_scales, value_scales, table, lens, starts=None, scale=None):
    """Attention in 64 bits over codes [pages, page_tokens, heads, dim] and
    scales [pages, blocks, heads]; NaN for tokens behind the last row's."""
    table, lens = _i32(table), _i32(lens)
    pages, page_tokens, heads, dim = keys.shape
    size = page_tokens // key_scales.shape[1]
    q = np.asarray(queries, np.float64)
    tokens, q_heads, _ = q.shape
    group = q_heads // heads
    out = np.full(q.shape, np.nan)
    f64p = ctypes.POINTER(ctypes.c_double)
    for s in range(lens.size):
        begin, n, first = _row_tokens(lens, starts, tokens, s)
        top = max(first + n, 0)
        at = np.arange(top)
        nth = at // page_tokens
        page = np.where(nth < table.shape[1], table[s, np.minimum(nth, max(table.shape[1] - 1, 0))]
                        if table.shape[1] else -1, -1)
        seen = ((page >= 0) & (page < pages)).astype(np.uint8)
        page, slot = np.where(seen > 0, page, 0), at % page_tokens
        if pages == 0:
            page, seen = page[:0], seen[:0]
            slot = slot[:0]
        for h in range(heads):
            kv = []
            for codes, scales in ((keys, key_scales), (values, value_scales)):
                x = code_values(codes[page, slot, h]).astype(np.float64)
                kv.append(np.ascontiguousarray(x * scales[page, slot // size, h].astype(np.float64)[:, None]))
            for i in range(n):
                m = min(max(first + i + 1, 0), len(seen))
                for j in range(h * group, (h + 1) * group):
                    x, o = np.ascontiguousarray(q[begin + i, j]), np.empty(dim)
                    _load().oracle_attend_query(x.ctypes.data_as(f64p), kv[0].ctypes.data_as(f64p),
                                                kv[1].ctypes.data_as(f64p), _up(seen), m, dim,
                                                dim**-0.5 if scale is None else scale, o.ctypes.data_as(f64p))
                    out[begin + i, j] = o
    return out
