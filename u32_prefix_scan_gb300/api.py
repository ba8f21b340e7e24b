"""Torch-tensor front end of libu32scan.so: argument marshalling only.

Every function takes CUDA tensors, checks dtype/device/contiguity, and
passes raw device pointers, sizes and the current CUDA stream to the C
entry point of the same name. All computation happens in the library's
kernels; nothing here touches tensor data.

U32 arrays are accepted as torch.int32 or torch.uint32 tensors (the bits are
the same; wrapping u32 addition and two's-complement int32 addition agree).

The library launches on the current device. sample_tokens, adjust_logits and
the pages_* calls refuse tensors, a stream or a workspace of another one.
"""

from __future__ import annotations

import functools
import threading

import torch

from . import _native

__all__ = [
    "Workspace",
    "scan_exclusive_u32",
    "scan_inclusive_u32",
    "scan_exclusive_u32_carry",
    "scan_inclusive_u32_carry",
    "reduce_u32_op",
    "count_nonzero_u32",
    "fill_splitmix_u32",
    "segscan_piece_summary_u32",
    "segscan_piece_carries_u32",
    "segscan_fix_u32",
    "compact_indices_u32_carry",
    "scan_exclusive_u32_host",
    "scan_inclusive_u32_host",
    "scan_u32_op",
    "scan_u64_op",
    "segscan_inclusive_u32",
    "segreduce_u32",
    "compact_indices_u32",
    "compact_values_u32",
    "radix_sort_perm_u32",
    "radix_sort_u32",
    "runs_layout_u32",
    "runs_owner_u32",
    "sample_tokens",
    "PagePool",
    "pages_copy",
    "pages_fork",
    "pages_free",
    "pages_compact",
    "adjust_logits",
    "KVCache",
    "pages_append",
    "pages_attend",
    "check",
]

_U32_DTYPES = (torch.int32, getattr(torch, "uint32", torch.int32))


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object around it


def _stream_handle(stream) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    if _raw_stream is None:
        return int(torch.cuda.current_stream().cuda_stream)
    return _raw_stream(torch.cuda.current_device())


def _launch_stream(stream, dev: int) -> int:
    """The handle of the stream for a call on tensors of CUDA device `dev`:
    the library launches on the current device, where another's pointers
    would fault."""
    current = torch.cuda.current_device()
    if dev != current:
        raise ValueError(f"the tensors are on cuda:{dev}, but cuda:{current} is current")
    if stream is not None and getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"stream must be on cuda:{dev}")
    return _stream_handle(stream)


def _require_cuda(t: torch.Tensor, name: str, dtypes=_U32_DTYPES) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class Workspace:
    """Device workspace for the library's carries, reused across calls.

    One zero-filled byte buffer per (device, stream), grown on demand. The
    library keeps it consistent between calls by itself; calls sharing a
    workspace must be ordered, which one stream guarantees.
    """

    _lock = threading.Lock()
    _cache: dict = {}

    def __init__(self, nbytes: int, device: torch.device):
        self.buf = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        self.ptr = self.buf.data_ptr()
        self.nbytes = self.buf.numel()

    @classmethod
    def get(cls, op: int, n: int, device: torch.device, stream_handle: int) -> "Workspace":
        need = _workspace_bytes(_native.lib(), op, n)
        key = (device.index, stream_handle)
        with cls._lock:
            ws = cls._cache.get(key)
            if ws is None or ws.nbytes < need:
                ws = cls(max(need, 2 * ws.nbytes if ws else need), device)
                current = torch.cuda.current_stream(device)
                if stream_handle != current.cuda_stream:  # filled on the current stream, used on the caller's
                    # (an ExternalStream of handle 0 would be some stream of torch's pool)
                    other = (torch.cuda.ExternalStream(stream_handle, device) if stream_handle
                             else torch.cuda.default_stream(device))
                    other.wait_stream(current)
                    ws.buf.record_stream(other)
                cls._cache[key] = ws
        return ws


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(lib, op: int, n: int) -> int:
    return lib.u32scan_workspace_bytes(op, n)


def _ws(op: int, n: int, device, stream_handle: int, workspace) -> Workspace:
    if workspace is not None:
        return workspace
    return Workspace.get(op, n, device, stream_handle)


def _scalar_out(out, like: torch.Tensor, dtype) -> torch.Tensor:
    if out is None:
        return torch.empty(1, dtype=dtype, device=like.device)
    _require_cuda(out, "out", (dtype,) if dtype not in _U32_DTYPES else _U32_DTYPES)
    if out.numel() < 1:
        raise ValueError("out must hold at least one element")
    return out


def _scan(name: str, data: torch.Tensor, total, stream, workspace) -> torch.Tensor:
    _require_cuda(data, "data")
    total = _scalar_out(total, data, data.dtype)
    n = data.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_SCAN, n, data.device, sh, workspace)
    fn = getattr(_native.lib(), name)
    _native.check(fn(data.data_ptr(), n, total.data_ptr(), ws.ptr, ws.nbytes, sh), name)
    return total


def scan_exclusive_u32(data: torch.Tensor, total: torch.Tensor | None = None, *, stream=None,
                       workspace: Workspace | None = None) -> torch.Tensor:
    """In place: data[j] <- data[0] + .. + data[j-1] (mod 2^32). Returns the
    one-element device tensor holding the wrapped total."""
    return _scan("scan_exclusive_u32", data, total, stream, workspace)


def scan_inclusive_u32(data: torch.Tensor, total: torch.Tensor | None = None, *, stream=None,
                       workspace: Workspace | None = None) -> torch.Tensor:
    """In place: data[j] <- data[0] + .. + data[j] (mod 2^32). Returns the
    one-element device tensor holding the wrapped total."""
    return _scan("scan_inclusive_u32", data, total, stream, workspace)


def _scan_carry(name: str, data: torch.Tensor, carry_in, total, stream, workspace) -> torch.Tensor:
    _require_cuda(data, "data")
    if carry_in is not None:
        _require_cuda(carry_in, "carry_in")
        if carry_in.numel() < 1:
            raise ValueError("carry_in must hold at least one element")
    total = _scalar_out(total, data, data.dtype)
    n = data.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_SCAN, n, data.device, sh, workspace)
    fn = getattr(_native.lib(), name)
    _native.check(fn(data.data_ptr(), n, carry_in.data_ptr() if carry_in is not None else None, total.data_ptr(),
                     ws.ptr, ws.nbytes, sh), name)
    return total


def scan_exclusive_u32_carry(data: torch.Tensor, carry_in: torch.Tensor | None, total: torch.Tensor | None = None,
                             *, stream=None, workspace: Workspace | None = None) -> torch.Tensor:
    """In place: data[j] <- carry_in + data[0] + .. + data[j-1] (mod 2^32),
    carry_in a one-element device tensor (None: 0). Returns the one-element
    device tensor holding carry_in + the wrapped sum of data."""
    return _scan_carry("scan_exclusive_u32_carry", data, carry_in, total, stream, workspace)


def scan_inclusive_u32_carry(data: torch.Tensor, carry_in: torch.Tensor | None, total: torch.Tensor | None = None,
                             *, stream=None, workspace: Workspace | None = None) -> torch.Tensor:
    """In place: data[j] <- carry_in + data[0] + .. + data[j] (mod 2^32).
    Returns carry_in + the wrapped sum of data (one-element device tensor)."""
    return _scan_carry("scan_inclusive_u32_carry", data, carry_in, total, stream, workspace)


def reduce_u32_op(data: torch.Tensor, op: str = "add", total: torch.Tensor | None = None, *, stream=None,
                  workspace: Workspace | None = None) -> torch.Tensor:
    """The fold of data under op in {add, mul, and, or, xor, min, max} (u32;
    add and mul wrap), read once. Returns a one-element device tensor."""
    if op not in _native.SCAN_OPS:
        raise ValueError(f"op must be one of {sorted(_native.SCAN_OPS)}")
    _require_cuda(data, "data")
    total = _scalar_out(total, data, data.dtype)
    n = data.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_REDUCE, n, data.device, sh, workspace)
    _native.check(_native.lib().reduce_u32_op(_native.SCAN_OPS[op], data.data_ptr(), n, total.data_ptr(), ws.ptr,
                                              ws.nbytes, sh), "reduce_u32_op")
    return total


def _require_pinned(t: torch.Tensor, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    # an empty tensor has no storage to pin and is never read
    if t.device.type != "cpu" or (t.numel() > 0 and not t.is_pinned()):
        raise ValueError(f"{name} must be a pinned (page-locked) CPU tensor")
    if t.dtype not in _U32_DTYPES:
        raise TypeError(f"{name} must have dtype in {_U32_DTYPES}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _scan_host(name: str, host_in: torch.Tensor, host_out, total, device, stream, workspace):
    _require_pinned(host_in, "host_in")
    if host_out is None:
        host_out = torch.empty_like(host_in).pin_memory()
    _require_pinned(host_out, "host_out")
    if host_out.numel() != host_in.numel():
        raise ValueError("host_in and host_out differ in length")
    if total is None:
        total = torch.empty(1, dtype=host_in.dtype).pin_memory()
    _require_pinned(total, "total")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    n = host_in.numel()
    with torch.cuda.device(device):
        sh = _stream_handle(stream)
        ws = _ws(_native.OP_SCAN_HOST, n, device, sh, workspace)
        fn = getattr(_native.lib(), name)
        _native.check(fn(host_in.data_ptr(), host_out.data_ptr(), n, total.data_ptr(), ws.ptr, ws.nbytes, sh), name)
    return host_out, total


def scan_exclusive_u32_host(host_in: torch.Tensor, host_out: torch.Tensor | None = None,
                            total: torch.Tensor | None = None, *, device=None, stream=None,
                            workspace: Workspace | None = None):
    """Exclusive scan of a pinned host array into a pinned host array (may be
    host_in itself), through the device. Asynchronous on the stream: the
    outputs are complete once the stream reaches the call. Returns
    (host_out, total), total a one-element pinned tensor."""
    return _scan_host("scan_exclusive_u32_host", host_in, host_out, total, device, stream, workspace)


def scan_inclusive_u32_host(host_in: torch.Tensor, host_out: torch.Tensor | None = None,
                            total: torch.Tensor | None = None, *, device=None, stream=None,
                            workspace: Workspace | None = None):
    """Inclusive scan of a pinned host array; otherwise as
    scan_exclusive_u32_host."""
    return _scan_host("scan_inclusive_u32_host", host_in, host_out, total, device, stream, workspace)


def scan_u32_op(data: torch.Tensor, op: str, inclusive: bool = False, total: torch.Tensor | None = None, *,
                stream=None, workspace: Workspace | None = None) -> torch.Tensor:
    """In place scan under op in {add, mul, and, or, xor, min, max} (u32;
    add and mul wrap). Returns the one-element device tensor holding the
    fold of all elements."""
    if op not in _native.SCAN_OPS:
        raise ValueError(f"op must be one of {sorted(_native.SCAN_OPS)}")
    _require_cuda(data, "data")
    total = _scalar_out(total, data, data.dtype)
    n = data.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_SCAN, n, data.device, sh, workspace)
    _native.check(_native.lib().scan_u32_op(_native.SCAN_OPS[op], int(bool(inclusive)), data.data_ptr(), n,
                                            total.data_ptr(), ws.ptr, ws.nbytes, sh), "scan_u32_op")
    return total


def scan_u64_op(data: torch.Tensor, op: str = "add", inclusive: bool = False, total: torch.Tensor | None = None,
                *, stream=None, workspace: Workspace | None = None) -> torch.Tensor:
    """In place scan of a 64-bit row (int64 or uint64 bits) under op in
    {add, mul, and, or, xor, min, max}, unsigned, add and mul wrapping at
    2^64. Returns the one-element device tensor holding the fold."""
    if op not in _native.SCAN_OPS:
        raise ValueError(f"op must be one of {sorted(_native.SCAN_OPS)}")
    u64 = (torch.int64, getattr(torch, "uint64", torch.int64))
    _require_cuda(data, "data", u64)
    if total is None:
        total = torch.empty(1, dtype=data.dtype, device=data.device)
    _require_cuda(total, "total", u64)
    n = data.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_SCAN64, n, data.device, sh, workspace)
    _native.check(_native.lib().scan_u64_op(_native.SCAN_OPS[op], int(bool(inclusive)), data.data_ptr(), n,
                                            total.data_ptr(), ws.ptr, ws.nbytes, sh), "scan_u64_op")
    return total


def _seg_args(data, head_flags, seg_sums, nseg):
    _require_cuda(data, "data")
    _require_cuda(head_flags, "head_flags", (torch.int32, torch.uint8))
    if head_flags.numel() != data.numel():
        raise ValueError("data and head_flags differ in length")
    if seg_sums is not None:
        _require_cuda(seg_sums, "seg_sums")
    nseg = _scalar_out(nseg, data, data.dtype)
    return nseg


def segscan_inclusive_u32(data: torch.Tensor, head_flags: torch.Tensor, seg_sums: torch.Tensor | None = None,
                          nseg: torch.Tensor | None = None, *, stream=None,
                          workspace: Workspace | None = None) -> torch.Tensor:
    """In place: data[j] <- sum of data over j's segment up to j (mod 2^32);
    a non-zero head flag (int32 or uint8) opens a segment, index 0 always does. If seg_sums
    is given, seg_sums[k] <- segment k's sum (for k < seg_sums.numel()).
    Returns the one-element device tensor holding the segment count."""
    nseg = _seg_args(data, head_flags, seg_sums, nseg)
    n = data.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_SEGSCAN, n, data.device, sh, workspace)
    name = "segscan_inclusive_u32" + ("_u8heads" if head_flags.dtype == torch.uint8 else "")
    _native.check(getattr(_native.lib(), name)(
        data.data_ptr(), head_flags.data_ptr(), n, seg_sums.data_ptr() if seg_sums is not None else None,
        seg_sums.numel() if seg_sums is not None else 0, nseg.data_ptr(), ws.ptr, ws.nbytes, sh), name)
    return nseg


def segreduce_u32(data: torch.Tensor, head_flags: torch.Tensor, seg_sums: torch.Tensor | None = None,
                  nseg: torch.Tensor | None = None, *, stream=None, workspace: Workspace | None = None):
    """Per-segment wrapped sums without writing the scan. seg_sums defaults
    to a fresh tensor of n elements (enough for any flag pattern). Returns
    (seg_sums, nseg): the first nseg entries of seg_sums are the sums."""
    if seg_sums is None:
        _require_cuda(data, "data")
        seg_sums = torch.empty(max(data.numel(), 1), dtype=data.dtype, device=data.device)
    nseg = _seg_args(data, head_flags, seg_sums, nseg)
    n = data.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_SEGSCAN, n, data.device, sh, workspace)
    name = "segreduce_u32" + ("_u8heads" if head_flags.dtype == torch.uint8 else "")
    _native.check(getattr(_native.lib(), name)(
        data.data_ptr(), head_flags.data_ptr(), n, seg_sums.data_ptr(), seg_sums.numel(), nseg.data_ptr(),
        ws.ptr, ws.nbytes, sh), name)
    return seg_sums, nseg


def compact_indices_u32(flags: torch.Tensor, offsets: torch.Tensor | None = None,
                        indices: torch.Tensor | None = None, count: torch.Tensor | None = None, *,
                        want_offsets: bool = True, stream=None, workspace: Workspace | None = None):
    """Stream compaction of int32 flags (non-zero keeps an element).
    Returns (offsets, indices, count): inclusive offsets (None when
    want_offsets is False and none were given), the kept indices at the
    front of `indices` with -1 after them, and the one-element count."""
    _require_cuda(flags, "flags", (torch.int32,))
    n = flags.numel()
    if offsets is None and want_offsets:
        offsets = torch.empty(n, dtype=torch.int32, device=flags.device)
    if offsets is not None:
        _require_cuda(offsets, "offsets", (torch.int32,))
        if offsets.numel() != n:
            raise ValueError("offsets must have n elements")
    if indices is None:
        indices = torch.empty(n, dtype=torch.int32, device=flags.device)
    _require_cuda(indices, "indices", (torch.int32,))
    if indices.numel() != n:
        raise ValueError("indices must have n elements")
    count = _scalar_out(count, flags, torch.int32)
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_COMPACT, n, flags.device, sh, workspace)
    _native.check(_native.lib().compact_indices_u32(
        flags.data_ptr(), n, offsets.data_ptr() if offsets is not None else None, indices.data_ptr(),
        count.data_ptr(), ws.ptr, ws.nbytes, sh), "compact_indices_u32")
    return offsets, indices, count


def compact_indices_u32_carry(flags: torch.Tensor, kept_before: torch.Tensor | None,
                              first_index: torch.Tensor | None, offsets: torch.Tensor | None = None,
                              indices: torch.Tensor | None = None, count: torch.Tensor | None = None, *,
                              stream=None, workspace: Workspace | None = None):
    """compact_indices_u32 of one piece of a longer flag array: kept_before
    and first_index (one-element int32 device tensors, or None for 0) are
    the kept elements and the elements before the piece. Returns (offsets,
    indices, count) as compact_indices_u32, with whole-array offsets and
    indices and the piece's own count."""
    _require_cuda(flags, "flags", (torch.int32,))
    for name, t in (("kept_before", kept_before), ("first_index", first_index)):
        if t is not None:
            _require_cuda(t, name, (torch.int32,))
            if t.numel() < 1:
                raise ValueError(f"{name} must hold at least one element")
    n = flags.numel()
    if offsets is None:
        offsets = torch.empty(n, dtype=torch.int32, device=flags.device)
    _require_cuda(offsets, "offsets", (torch.int32,))
    if indices is None:
        indices = torch.empty(n, dtype=torch.int32, device=flags.device)
    _require_cuda(indices, "indices", (torch.int32,))
    if offsets.numel() != n or indices.numel() != n:
        raise ValueError("offsets and indices must have n elements")
    count = _scalar_out(count, flags, torch.int32)
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_COMPACT, n, flags.device, sh, workspace)
    _native.check(_native.lib().compact_indices_u32_carry(
        flags.data_ptr(), n, kept_before.data_ptr() if kept_before is not None else None,
        first_index.data_ptr() if first_index is not None else None, offsets.data_ptr(), indices.data_ptr(),
        count.data_ptr(), ws.ptr, ws.nbytes, sh), "compact_indices_u32_carry")
    return offsets, indices, count


def segscan_piece_summary_u32(scanned: torch.Tensor, head_flags: torch.Tensor, nseg: torch.Tensor,
                              first_opens: bool, summary: torch.Tensor | None = None, *,
                              stream=None) -> torch.Tensor:
    """A piece's summary after segscan_inclusive_u32: (has head, tail,
    segments starting in it), three words in a device tensor."""
    _require_cuda(scanned, "scanned")
    _require_cuda(head_flags, "head_flags", (torch.int32,))
    _require_cuda(nseg, "nseg")
    if head_flags.numel() != scanned.numel():
        raise ValueError("head_flags must have as many elements as scanned")
    if summary is None:
        summary = torch.empty(3, dtype=torch.int32, device=scanned.device)
    _require_cuda(summary, "summary")
    if summary.numel() < 3:
        raise ValueError("summary must hold three elements")
    _native.check(_native.lib().segscan_piece_summary_u32(
        scanned.data_ptr(), head_flags.data_ptr(), scanned.numel(), nseg.data_ptr(), int(bool(first_opens)),
        summary.data_ptr(), _stream_handle(stream)), "segscan_piece_summary_u32")
    return summary


def segscan_piece_carries_u32(summaries: torch.Tensor, carries: torch.Tensor | None = None,
                              nseg_total: torch.Tensor | None = None, *, stream=None):
    """From g pieces' summaries (3 g words, in piece order): each piece's
    carry-in and the whole array's segment count (device tensors)."""
    _require_cuda(summaries, "summaries")
    if summaries.numel() % 3:
        raise ValueError("summaries must hold three words a piece")
    g = summaries.numel() // 3
    if carries is None:
        carries = torch.empty(g, dtype=torch.int32, device=summaries.device)
    _require_cuda(carries, "carries")
    nseg_total = _scalar_out(nseg_total, summaries, torch.int32)
    _native.check(_native.lib().segscan_piece_carries_u32(summaries.data_ptr(), g, carries.data_ptr(),
                                                          nseg_total.data_ptr(), _stream_handle(stream)),
                  "segscan_piece_carries_u32")
    return carries, nseg_total


def segscan_fix_u32(data: torch.Tensor, head_flags: torch.Tensor, carry: torch.Tensor, *, stream=None,
                    workspace: Workspace | None = None) -> torch.Tensor:
    """Adds carry (one-element device tensor) to the elements of the scanned
    piece before its first head. Returns data."""
    _require_cuda(data, "data")
    _require_cuda(head_flags, "head_flags", (torch.int32,))
    _require_cuda(carry, "carry")
    if head_flags.numel() != data.numel():
        raise ValueError("head_flags must have as many elements as data")
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_REDUCE, data.numel(), data.device, sh, workspace)
    _native.check(_native.lib().segscan_fix_u32(data.data_ptr(), head_flags.data_ptr(), data.numel(),
                                                carry.data_ptr(), ws.ptr, ws.nbytes, sh), "segscan_fix_u32")
    return data


def count_nonzero_u32(data: torch.Tensor, count: torch.Tensor | None = None, *, stream=None,
                      workspace: Workspace | None = None) -> torch.Tensor:
    """The number of non-zero elements of data (u32 or int32 flags), read
    once. Returns a one-element device tensor."""
    _require_cuda(data, "data")
    count = _scalar_out(count, data, data.dtype)
    n = data.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_REDUCE, n, data.device, sh, workspace)
    _native.check(_native.lib().count_nonzero_u32(data.data_ptr(), n, count.data_ptr(), ws.ptr, ws.nbytes, sh),
                  "count_nonzero_u32")
    return count


def fill_splitmix_u32(n: int, seed: int, stream_id: int = 0, start: int = 0, *, device=None,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The seeded input u32(seed, stream_id, start + i), i < n, drawn on the
    device: the same numbers as inputs.splitmix_u32 (counter-based
    SplitMix64), without a copy from the host. Returns an int32 tensor
    holding the u32 bits (out, when given, is filled and returned)."""
    if out is None:
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        out = torch.empty(n, dtype=torch.int32, device=dev)
    _require_cuda(out, "out")
    if out.numel() != n:
        raise ValueError("out must hold n elements")
    sh = _stream_handle(stream)
    _native.check(_native.lib().u32scan_fill_splitmix_u32(out.data_ptr(), n, seed, stream_id, start, sh),
                  "u32scan_fill_splitmix_u32")
    return out


def compact_values_u32(values: torch.Tensor, flags: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       count: torch.Tensor | None = None, *, stream=None, workspace: Workspace | None = None):
    """The kept values, in order, at the front of `out` (the rest of out is
    left as it was); an element is kept when its flag is non-zero, or, with
    no flags, when its value is. Returns (out, count)."""
    _require_cuda(values, "values")
    n = values.numel()
    if flags is not None:
        _require_cuda(flags, "flags", (torch.int32,))
        if flags.numel() != n:
            raise ValueError("values and flags differ in length")
    if out is None:
        out = torch.empty_like(values)
    _require_cuda(out, "out")
    if out.numel() != n:
        raise ValueError("out must have n elements")
    count = _scalar_out(count, values, torch.int32)
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_COMPACT, n, values.device, sh, workspace)
    _native.check(_native.lib().compact_values_u32(values.data_ptr(), flags.data_ptr() if flags is not None else None,
                                                   n, out.data_ptr(), count.data_ptr(), ws.ptr, ws.nbytes, sh),
                  "compact_values_u32")
    return out, count


def radix_sort_perm_u32(keys: torch.Tensor, perm: torch.Tensor | None = None, *, stream=None,
                        workspace: Workspace | None = None) -> torch.Tensor:
    """The stable sorting permutation of u32 keys (int32 or uint32 tensor,
    unsigned order): keys[perm] is non-decreasing, ties by index."""
    _require_cuda(keys, "keys")
    n = keys.numel()
    if perm is None:
        perm = torch.empty(n, dtype=torch.int32, device=keys.device)
    _require_cuda(perm, "perm", (torch.int32,))
    if perm.numel() != n:
        raise ValueError("perm must have n elements")
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_RADIX, n, keys.device, sh, workspace)
    _native.check(_native.lib().radix_sort_perm_u32(keys.data_ptr(), n, perm.data_ptr(), ws.ptr, ws.nbytes, sh),
                  "radix_sort_perm_u32")
    return perm


def radix_sort_u32(keys: torch.Tensor, keys_out: torch.Tensor | None = None, perm: torch.Tensor | None = None,
                   *, want_perm: bool = True, stream=None, workspace: Workspace | None = None):
    """Stable radix sort of u32 keys (unsigned order). Returns (keys_out,
    perm): the sorted keys and, unless want_perm is False and no perm was
    given, the stable permutation (keys_out = keys[perm])."""
    _require_cuda(keys, "keys")
    n = keys.numel()
    if keys_out is None:
        keys_out = torch.empty_like(keys)
    _require_cuda(keys_out, "keys_out")
    if keys_out.numel() != n:
        raise ValueError("keys_out must have n elements")
    if perm is None and want_perm:
        perm = torch.empty(n, dtype=torch.int32, device=keys.device)
    if perm is not None:
        _require_cuda(perm, "perm", (torch.int32,))
        if perm.numel() != n:
            raise ValueError("perm must have n elements")
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_RADIX, n, keys.device, sh, workspace)
    _native.check(_native.lib().radix_sort_u32(keys.data_ptr(), n, keys_out.data_ptr(),
                                               perm.data_ptr() if perm is not None else None, ws.ptr, ws.nbytes, sh),
                  "radix_sort_u32")
    return keys_out, perm


def runs_layout_u32(counts: torch.Tensor, entries: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                    *, stream=None, workspace: Workspace | None = None) -> torch.Tensor:
    """In place: counts[i] <- ends[i] = counts[0] + .. + counts[i] (mod
    2^32). Returns the one-element device tensor entries = max(total, 1);
    when given, slots[0 : min(entries, slots.numel())] is set to -1."""
    _require_cuda(counts, "counts")
    entries = _scalar_out(entries, counts, counts.dtype)
    if slots is not None:
        _require_cuda(slots, "slots", (torch.int32,))
    n = counts.numel()
    sh = _stream_handle(stream)
    ws = _ws(_native.OP_RUNS, n, counts.device, sh, workspace)
    _native.check(_native.lib().runs_layout_u32(counts.data_ptr(), n, entries.data_ptr(),
                                                slots.data_ptr() if slots is not None else None,
                                                slots.numel() if slots is not None else 0, ws.ptr, ws.nbytes, sh),
                  "runs_layout_u32")
    return entries


def runs_owner_u32(ends: torch.Tensor, owner: torch.Tensor | None = None, capacity: int | None = None, *,
                   stream=None) -> torch.Tensor:
    """owner[e] = the owner whose run holds entry e (the least i with
    e < ends[i]) for e in [0, min(entries, capacity)); -1 for the one slot of
    an empty layout. With no `owner` tensor, one of `capacity` elements is
    made (capacity defaults to entries, read back from the device)."""
    _require_cuda(ends, "ends")
    n = ends.numel()
    if owner is None:
        if capacity is None:
            total = int(ends[-1].item()) & 0xFFFFFFFF if n else 0
            capacity = max(total, 1)
        owner = torch.empty(capacity, dtype=torch.int32, device=ends.device)
    _require_cuda(owner, "owner", (torch.int32,))
    cap = owner.numel() if capacity is None else min(int(capacity), owner.numel())
    sh = _stream_handle(stream)
    _native.check(_native.lib().runs_owner_u32(ends.data_ptr(), n, owner.data_ptr(), cap, sh), "runs_owner_u32")
    return owner


def _new(n, dtype, device: torch.device, stream) -> torch.Tensor:
    """An output (of n elements or shape n) for a call on `stream`, in memory of that stream: what the
    current one gave back may still be in use there. The caller goes on with
    it on the current stream, so that one is noted too."""
    if stream is None or stream.cuda_stream == _stream_handle(None):
        return torch.empty(n, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = torch.empty(n, dtype=dtype, device=device)
    out.record_stream(current)
    return out


_LOGIT_TYPES = {torch.float32: _native.F32, torch.float16: _native.F16, torch.bfloat16: _native.BF16}


def _tensor(t, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _misplaced(t, name: str, dev: int) -> ValueError:
    if not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    return ValueError(f"{name} must be on cuda:{dev}")


def _arg(t, name: str, dtype, numel: int, dev: int) -> int:
    """The device pointer of a contiguous tensor of at least numel elements
    on CUDA device `dev`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise _misplaced(t, name, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise _misplaced(t, name, dev)
    if t.numel() < numel:
        raise ValueError(f"{name} must hold at least {numel} elements")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _optional(t, name: str, dtype, numel: int, dev: int) -> int | None:
    return None if t is None else _arg(t, name, dtype, numel, dev)


def sample_tokens(logits: torch.Tensor, random: torch.Tensor, *, temperature: torch.Tensor | None = None,
                  top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                  min_p: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                  probs: torch.Tensor | None = None, stream=None):
    """The next token of every row of logits [rows, vocab] (float32, float16
    or bfloat16; rows may be strided, elements of a row are adjacent), drawn
    with the u32 words random [rows]. temperature, top_p, min_p (float32) and
    top_k (int32) hold one value a row; None is temperature 1 and no filter.
    Returns (tokens, probs): int32 tokens, -1 where every logit is -inf or
    NaN, and the chosen tokens' probabilities after the filters. The result
    is exact: integer weights, sums and draw, as include/u32scan.h states
    them."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor (this library has no CPU path)")
    kind = _LOGIT_TYPES.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must have dtype in {tuple(_LOGIT_TYPES)}, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must have two dimensions, [rows, vocab]")
    rows, vocab = logits.shape
    row_stride, step = logits.stride()
    if step != 1 and vocab > 1 and rows > 0:
        raise ValueError("the elements of a row of logits must be adjacent")
    dev = logits.get_device()
    sh = _launch_stream(stream, dev)
    if tokens is None:
        tokens = _new(rows, torch.int32, logits.device, stream)
    if probs is None:
        probs = _new(rows, torch.float32, logits.device, stream)
    f32, i32 = torch.float32, torch.int32
    words = _arg(random, "random", i32 if _tensor(random, "random").dtype is i32 else _U32_DTYPES[1], rows, dev)
    _native.check(_native.lib().sample_tokens(
        logits.data_ptr(), kind, rows, vocab, row_stride, _optional(temperature, "temperature", f32, rows, dev),
        _optional(top_k, "top_k", i32, rows, dev), _optional(top_p, "top_p", f32, rows, dev),
        _optional(min_p, "min_p", f32, rows, dev), words, _arg(tokens, "tokens", i32, rows, dev),
        _arg(probs, "probs", f32, rows, dev), sh), "sample_tokens")
    return tokens, probs


class PagePool:
    """The planes of a paged cache, for the pages_* calls.

    tensors: one CUDA tensor a plane, [pages, ...] (say, each layer's keys
    and each layer's values), all of one shape, dtype and strides, with a
    page's elements adjacent; or, with planes_first, one tensor [planes,
    pages, ...]. The pool keeps the tensors alive and their addresses in
    device memory; make it once per cache.
    """

    def __init__(self, tensors, *, planes_first: bool = False):
        if isinstance(tensors, torch.Tensor):
            if planes_first and tensors.dim() < 2:
                raise ValueError("a tensor with its planes first must have at least two dimensions")
            tensors = list(tensors.unbind(0)) if planes_first else [tensors]
        tensors = list(tensors)
        if not tensors:
            raise ValueError("a pool needs at least one plane")
        first = tensors[0]
        for t in tensors:
            if not isinstance(t, torch.Tensor):
                raise TypeError("a pool's planes must be torch tensors")
            if t.device.type != "cuda":
                raise ValueError("a pool's planes must be CUDA tensors (this library has no CPU path)")
            if (t.dim() < 1 or t.shape != first.shape or t.stride() != first.stride() or t.dtype != first.dtype
                    or t.device != first.device):
                raise ValueError("a pool's planes must agree in shape, strides, dtype and device")
        item = first.element_size()
        self.pages = first.shape[0]
        self.page_bytes = item
        for d in first.shape[1:]:
            self.page_bytes *= d
        if self.pages > 0 and not first[0].is_contiguous():
            raise ValueError("a page's elements must be adjacent")
        self.page_stride = first.stride(0) * item if self.pages > 1 else self.page_bytes
        if self.page_stride < self.page_bytes:
            raise ValueError("a pool's pages must not overlap")
        self.tensors = tensors
        self.device = first.device
        self._planes = torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64, device=self.device)
        torch.cuda.current_stream(self.device).synchronize()  # the addresses may be read on any stream
        self.struct = _native.PagePoolStruct(self._planes.data_ptr(), len(tensors), self.pages, self.page_bytes,
                                             self.page_stride)


def _pool_struct(pool, dev: int):
    if not isinstance(pool, PagePool):
        raise TypeError("pool must be a PagePool")
    if pool.device.index != dev:
        raise ValueError(f"pool must be on cuda:{dev}")
    return pool.struct


def pages_copy(pool: PagePool, src: torch.Tensor, dst: torch.Tensor, count: torch.Tensor | None = None, *,
               stream=None) -> None:
    """Copies page src[i] to page dst[i] in every plane of the pool (int32
    tensors; pairs with a number outside the pool are skipped; no page may
    be a destination twice, or both a destination and another pair's
    source). count, a one-element int32 tensor, limits the pairs on the
    device."""
    struct, i32 = _pool_struct(pool, pool.device.index if isinstance(pool, PagePool) else -1), torch.int32
    dev, n = pool.device.index, _tensor(src, "src").numel()
    sh = _launch_stream(stream, dev)
    if _tensor(dst, "dst").numel() != n:
        raise ValueError("src and dst differ in length")
    _native.check(_native.lib().pages_copy(struct, _arg(src, "src", i32, n, dev), _arg(dst, "dst", i32, n, dev), n,
                                           _optional(count, "count", i32, 1, dev), sh), "pages_copy")


def _cache_args(table, lens, refs, page_tokens):
    """The checked leading arguments of the calls on a paged cache, and their
    device."""
    if not isinstance(table, torch.Tensor):
        raise TypeError("table must be a torch.Tensor")
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor (this library has no CPU path)")
    if table.dtype is not torch.int32:
        raise TypeError(f"table must have dtype torch.int32, got {table.dtype}")
    if table.dim() != 2:
        raise ValueError("table must have two dimensions, [rows, width]")
    rows, width = table.shape
    stride, step = table.stride()
    if rows == 0:
        stride = width
    elif step != 1 and width > 1:
        raise ValueError("the entries of a row of table must be adjacent")
    elif rows == 1:
        stride = width
    elif stride < width:
        raise ValueError("the rows of table must not overlap")
    dev = table.get_device()
    lens_ptr, refs_ptr = _arg(lens, "lens", torch.int32, rows, dev), _arg(refs, "refs", torch.int32, 0, dev)
    if lens.numel() != rows:
        raise ValueError("lens must hold one length for every row of table")
    return (table.data_ptr(), stride, rows, width, lens_ptr, refs_ptr, refs.numel(), page_tokens), dev


def _pages_ws(args, table, dev: int, sh: int, workspace) -> Workspace:
    if workspace is None:
        return Workspace.get(_native.OP_PAGES, args[6] + args[2], table.device, sh)
    if workspace.buf.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev}")
    return workspace


def _one_out(out, name: str, like: torch.Tensor, dev: int, stream) -> tuple[torch.Tensor, int]:
    if out is None:
        out = _new(1, torch.int32, like.device, stream)
    return out, _arg(out, name, torch.int32, 1, dev)


def pages_fork(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_tokens: int, *,
               parent: torch.Tensor | None = None, grow: torch.Tensor | None = None, pool: PagePool | None = None,
               status: torch.Tensor | None = None, free_pages: torch.Tensor | None = None, stream=None,
               workspace: Workspace | None = None):
    """Forks rows and gives rows their next pages, in place. Empty rows s
    with parent[s] >= 0 become copies of that row (full pages shared, a
    partly filled last one copied in the pool); then every row grows by
    grow[s] tokens. Fresh pages are the free ones (refs = 0) in ascending
    order, dealt in row order. Returns (status, free_pages): per row the
    fresh pages taken, -1 (refused) or -2 (out of pages; the row is left as
    it was), and the number of free pages left."""
    args, dev = _cache_args(table, lens, refs, page_tokens)
    sh = _launch_stream(stream, dev)
    rows, i32 = args[2], torch.int32
    if status is None:
        status = _new(rows, i32, table.device, stream)
    free_pages, free_ptr = _one_out(free_pages, "free_pages", table, dev, stream)
    ws = _pages_ws(args, table, dev, sh, workspace)
    _native.check(_native.lib().pages_fork(
        *args, _optional(parent, "parent", i32, rows, dev), _optional(grow, "grow", i32, rows, dev),
        None if pool is None else _pool_struct(pool, dev), _arg(status, "status", i32, rows, dev), free_ptr, ws.ptr,
        ws.nbytes, sh), "pages_fork")
    return status, free_pages


def pages_free(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_tokens: int, release: torch.Tensor,
               *, freed: torch.Tensor | None = None, stream=None, workspace: Workspace | None = None) -> torch.Tensor:
    """Releases, in place, every row s with release[s] != 0 (int32): its
    pages' refs fall by one, its entries become -1, its length 0. Returns the
    number of pages that became free (one-element device tensor)."""
    args, dev = _cache_args(table, lens, refs, page_tokens)
    sh = _launch_stream(stream, dev)
    freed, freed_ptr = _one_out(freed, "freed", table, dev, stream)
    ws = _pages_ws(args, table, dev, sh, workspace)
    _native.check(_native.lib().pages_free(*args, _arg(release, "release", torch.int32, args[2], dev), freed_ptr,
                                           ws.ptr, ws.nbytes, sh), "pages_free")
    return freed


def pages_compact(pool: PagePool | None, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                  page_tokens: int, *, live: torch.Tensor | None = None, remap: torch.Tensor | None = None,
                  stream=None, workspace: Workspace | None = None):
    """Packs the live pages (refs != 0) into the first ones, in place: those
    past the number L of live pages move, in order, into the free pages
    below L; table and refs follow. Returns (live, remap): L, and each live
    page's new number (-1 for free ones)."""
    args, dev = _cache_args(table, lens, refs, page_tokens)
    sh = _launch_stream(stream, dev)
    pages = args[6]
    live, live_ptr = _one_out(live, "live", table, dev, stream)
    if remap is None:
        remap = _new(pages, torch.int32, table.device, stream)
    ws = _pages_ws(args, table, dev, sh, workspace)
    _native.check(_native.lib().pages_compact(
        None if pool is None else _pool_struct(pool, dev), *args, live_ptr,
        _arg(remap, "remap", torch.int32, pages, dev), ws.ptr, ws.nbytes, sh), "pages_compact")
    return live, remap


def _matrix(t, name: str, dtypes, rows: int, dev: int) -> tuple[int, int, int]:
    """Pointer, width and row stride of a tensor [rows, width] whose rows'
    elements are adjacent; zeros for None."""
    if t is None:
        return 0, 0, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        if not t.is_cuda:
            raise _misplaced(t, name, dev)
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if t.get_device() != dev:
        raise _misplaced(t, name, dev)
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows:
        raise ValueError(f"{name} must have two dimensions, the first of {rows}")
    stride, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent")
    return t.data_ptr(), shape[1], stride


def adjust_logits(logits: torch.Tensor, *, history: torch.Tensor | None = None,
                  history_lens: torch.Tensor | None = None, prompt_lens: torch.Tensor | None = None,
                  repetition: torch.Tensor | None = None, presence: torch.Tensor | None = None,
                  frequency: torch.Tensor | None = None, bias_tokens: torch.Tensor | None = None,
                  bias: torch.Tensor | None = None, allowed: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """A request's rules applied to every row of logits [rows, vocab]
    (float32, float16 or bfloat16; rows may be strided) before sample_tokens.

    history [rows, width] (int32) holds each row's tokens, history_lens of them
    (None: width), the first prompt_lens (None: 0) its prompt; tokens outside
    the vocabulary are skipped. A token that occurs in it is divided by
    repetition where its logit is above 0 and multiplied by it elsewhere; one
    that occurs c times past the prompt loses frequency * c, then presence
    (float32, one value a row). bias_tokens, bias [rows, n] (int32, float32) add
    to the tokens they name (of a token named twice the last counts). A token whose bit in
    allowed [rows, ceil(vocab / 32)] (int32 or uint32; token 32 w + j is bit j of
    word w) is 0 becomes -inf.

    Returns out, a new tensor unless one is given; out=logits works in place.
    Exact: f32 operations in this order, each rounded alone, then rounded to
    the type."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor (this library has no CPU path)")
    kind = _LOGIT_TYPES.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must have dtype in {tuple(_LOGIT_TYPES)}, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must have two dimensions, [rows, vocab]")
    rows, vocab = logits.shape
    row_stride, step = logits.stride()
    if step != 1 and vocab > 1 and rows > 0:
        raise ValueError("the elements of a row of logits must be adjacent")
    dev = logits.get_device()
    sh = _launch_stream(stream, dev)
    if out is None:
        out = _new((rows, vocab), logits.dtype, logits.device, stream)
        out_ptr, out_stride = out.data_ptr(), vocab
    else:
        out_ptr, width, out_stride = _matrix(out, "out", (logits.dtype,), rows, dev)
        if width != vocab:
            raise ValueError("out must have the shape of logits")
    f32, i32 = torch.float32, torch.int32
    bias_ptr, biases, _ = _matrix(bias, "bias", (f32,), rows, dev)
    named = _arg(bias_tokens, "bias_tokens", i32, rows * biases, dev) if bias is not None else 0
    if bias is None and bias_tokens is not None:
        raise ValueError("bias_tokens needs bias")
    if bias is not None and (not bias.is_contiguous() or bias_tokens.shape != bias.shape):
        raise ValueError("bias_tokens and bias must be contiguous and agree in shape")
    history_ptr, held, history_stride = _matrix(history, "history", (i32,), rows, dev)
    mask_ptr, words, mask_stride = _matrix(allowed, "allowed", _U32_DTYPES, rows, dev)
    if allowed is not None and words != (vocab + 31) // 32:
        raise ValueError("allowed must have ceil(vocab / 32) words a row")
    rules = _native.pack_logit_rules(
        history_ptr, held, history_stride, _optional(history_lens, "history_lens", i32, rows, dev) or 0,
        _optional(prompt_lens, "prompt_lens", i32, rows, dev) or 0, _optional(repetition, "repetition", f32, rows, dev) or 0,
        _optional(presence, "presence", f32, rows, dev) or 0, _optional(frequency, "frequency", f32, rows, dev) or 0, named,
        bias_ptr, biases, mask_ptr, mask_stride)
    _native.check(_native.lib().adjust_logits(logits.data_ptr(), kind, rows, vocab, row_stride, out_ptr, out_stride,
                                              rules, sh), "adjust_logits")
    return out


_CACHE_TYPES = {**_LOGIT_TYPES, torch.float8_e4m3fn: _native.E4M3}


def _meet(apart: int, axes, run: int) -> bool:
    """Whether two arrays of the same nested strides, `apart` elements from
    each other, share one: axes (stride, size), the widest first, over runs of
    adjacent elements."""
    if not axes:
        return abs(apart) < run
    (stride, n), rest = axes[0], axes[1:]
    nearest = apart // stride  # (what the rest adds is less than a stride, up or down)
    return any(abs(k) < n and _meet(apart - k * stride, rest, run) for k in (nearest, nearest + 1))


class KVCache:
    """One layer's keys and values in a paged cache, for pages_append and
    pages_attend.

    keys, values: CUDA tensors [pages, page_tokens, heads, dim] of one shape,
    dtype (float32, float16, bfloat16 or float8_e4m3fn) and strides, with a
    head's elements adjacent; views of a PagePool's planes, say. With
    float8_e4m3fn, key_scales and value_scales (float32 [pages, blocks, heads],
    a page's scales adjacent, one stride for both) hold a scale for every
    block of page_tokens / blocks tokens and head: a value is its code times
    its scale. To let the pages_* calls move scales with their codes, make
    both views of one page of bytes. Keeps the tensors alive; make it once a
    layer. One whose keys and values (or their scales) share memory can be
    read, but not appended to.
    """

    def __init__(self, keys: torch.Tensor, values: torch.Tensor, key_scales: torch.Tensor | None = None,
                 value_scales: torch.Tensor | None = None):
        for name, t in (("keys", keys), ("values", values)):
            if not _tensor(t, name).is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
            if t.dtype not in _CACHE_TYPES:
                raise TypeError(f"{name} must have dtype in {tuple(_CACHE_TYPES)}, got {t.dtype}")
            if t.dim() != 4:
                raise ValueError(f"{name} must have four dimensions, [pages, page_tokens, heads, dim]")
        self.device = keys.device
        if (keys.shape != values.shape or keys.stride() != values.stride() or keys.dtype != values.dtype
                or keys.device != values.device):
            raise ValueError("keys and values must agree in shape, strides, dtype and device")
        if keys.stride(3) != 1 and keys.shape[3] > 1:
            raise ValueError("the elements of a head must be adjacent")
        pages, page_tokens, heads, dim = keys.shape
        if 0 in (page_tokens, heads, dim):
            raise ValueError("a cache needs tokens, heads and dimensions")
        # sizes of which there is one need no stride, and torch keeps any there
        strides = [s if n > 1 else 0 for s, n in zip(keys.stride()[:3], keys.shape[:3])]
        spans = sorted((s, n) for s, n in zip(strides, keys.shape[:3]) if n > 1)
        reach = dim
        for s, n in spans:
            if s < reach:
                raise ValueError("a cache's elements must not overlap")
            reach = s * (n - 1) + reach
        apart = values.data_ptr() - keys.data_ptr()
        self.shared = pages > 0 and _meet(apart // keys.element_size(), spans[::-1], dim)
        coded = keys.dtype is torch.float8_e4m3fn
        if coded != (key_scales is not None) or coded != (value_scales is not None):
            raise ValueError("key_scales and value_scales belong to a cache of float8_e4m3fn")
        blocks = scale_stride = 0
        if coded:
            for name, t in (("key_scales", key_scales), ("value_scales", value_scales)):
                if not _tensor(t, name).is_cuda or t.device != self.device:
                    raise ValueError(f"{name} must be on the keys' device")
                if t.dtype is not torch.float32:
                    raise TypeError(f"{name} must have dtype torch.float32, got {t.dtype}")
                if t.dim() != 3 or t.shape[0] != pages or t.shape[2] != heads:
                    raise ValueError(f"{name} must have the shape [pages, blocks, heads]")
                if pages > 0 and not t[0].is_contiguous():
                    raise ValueError(f"a page's {name} must be adjacent")
            blocks = key_scales.shape[1]
            if value_scales.shape != key_scales.shape or (pages > 1 and value_scales.stride(0) != key_scales.stride(0)):
                raise ValueError("key_scales and value_scales must agree in shape and strides")
            if blocks == 0 or page_tokens % blocks:
                raise ValueError("a page's tokens must fall into equal blocks")
            scale_stride = key_scales.stride(0) if pages > 1 else 0
            if pages > 1 and scale_stride < blocks * heads:
                raise ValueError("a cache's scales must not overlap")
            apart = value_scales.data_ptr() - key_scales.data_ptr()
            self.shared |= pages > 0 and _meet(apart // 4, [(scale_stride, pages)] if pages > 1 else [], blocks * heads)
        self.keys, self.values, self.key_scales, self.value_scales = keys, values, key_scales, value_scales
        self.dtype, self.heads, self.dim = keys.dtype, heads, dim
        self.struct = _native.KVCacheStruct(
            keys.data_ptr(), values.data_ptr(), _CACHE_TYPES[keys.dtype], pages, page_tokens, heads, dim, *strides,
            key_scales.data_ptr() if coded else None, value_scales.data_ptr() if coded else None, blocks, scale_stride)


def _cache_rows(cache, table, lens, starts, tokens: int):
    """The checked leading arguments of the calls on a KVCache, and their
    device."""
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    dev = cache.device.index
    ptr, width, stride = _matrix(_tensor(table, "table"), "table", (torch.int32,), table.shape[0] if table.dim() else 0,
                                 dev)
    rows = table.shape[0]
    if rows <= 1:
        stride = width
    elif stride < width:
        raise ValueError("the rows of table must not overlap")
    lens_ptr = _arg(lens, "lens", torch.int32, rows, dev)
    if lens.numel() != rows:
        raise ValueError("lens must hold one length for every row of table")
    if starts is not None:
        starts_ptr = _arg(starts, "starts", torch.int32, rows + 1, dev)
    elif tokens != rows:
        raise ValueError("without starts there must be one token for every row of table")
    else:
        starts_ptr = None
    return cache.struct, ptr, stride, rows, width, lens_ptr, starts_ptr


def _heads_arg(t, name: str, dtype, tokens: int, heads: int | None, dim: int, dev: int):
    """Pointer and strides of a tensor [tokens, heads, dim] whose heads'
    elements are adjacent."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        if not t.is_cuda:
            raise _misplaced(t, name, dev)
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise _misplaced(t, name, dev)
    shape = t.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have the shape [{tokens}, {'heads' if heads is None else heads}, {dim}]")
    token_stride, head_stride, step = t.stride()
    if step != 1 and dim > 1 and t.numel():
        raise ValueError(f"the elements of a head of {name} must be adjacent")
    return t.data_ptr(), token_stride if tokens > 1 else 0, head_stride if shape[1] > 1 else 0


def _distinct(t, name: str) -> None:
    """Refuses an output whose elements share memory (heads and tokens in
    either order)."""
    if t.is_contiguous():
        return
    (tokens, heads, dim), (token_stride, head_stride, _) = t.shape, t.stride()
    reach = dim
    for stride, n in sorted(((token_stride, tokens), (head_stride, heads))):
        if n > 1 and stride < reach and t.numel():
            raise ValueError(f"the heads of {name} must not overlap")
        if n > 1:
            reach += stride * (n - 1)


def pages_append(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, new_keys: torch.Tensor,
                 new_values: torch.Tensor, *, starts: torch.Tensor | None = None, status: torch.Tensor | None = None,
                 cos: torch.Tensor | None = None, sin: torch.Tensor | None = None, interleaved: bool = False,
                 queries: torch.Tensor | None = None, queries_out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor | None:
    """Writes new keys and values [tokens, heads, dim] (float32, float16 or
    bfloat16) into the pages that pages_fork gave their rows, keys rotated by
    their position on the way, and returns the rotated queries.

    Row s has the tokens starts[s] .. starts[s + 1] - 1 (int32 [rows + 1];
    None: one token a row), the last of its lens[s]. cos, sin (float32
    [positions, pairs]) hold each position's angles; element i of a head pairs
    with pairs + i, or 2 i with 2 i + 1 when interleaved, and elements from 2
    pairs on stay. A cache of float8_e4m3fn gets a power of two for every
    block's scale, the least under which the block's largest magnitude fits;
    when new tokens raise the scale of a block that holds older ones, those are
    rounded to it. Other caches have the tokens' dtype.

    Rows with status[s] < 0 (pages_fork's answer) are left as they were, and so
    are tokens whose position has no page or no angles; tokens behind the
    last row's are ignored. queries [tokens, q_heads, dim], rotated likewise,
    go to queries_out (a new tensor by default; queries itself works in place,
    other memory of queries, new_keys or new_values does not)."""
    tokens = new_keys.shape[0] if _tensor(new_keys, "new_keys").dim() else 0
    args = _cache_rows(cache, table, lens, starts, tokens)
    if cache.shared:
        raise ValueError("the cache's keys and values share memory: it can only be read")
    dev, heads, dim = cache.device.index, cache.heads, cache.dim
    sh = _launch_stream(stream, dev)
    dtype = new_keys.dtype
    kind = _LOGIT_TYPES.get(dtype)
    if kind is None:
        raise TypeError(f"new_keys must have dtype in {tuple(_LOGIT_TYPES)}, got {dtype}")
    if cache.dtype is not torch.float8_e4m3fn and cache.dtype is not dtype:
        raise TypeError(f"new_keys must have the cache's dtype {cache.dtype}, got {dtype}")
    k = _heads_arg(new_keys, "new_keys", dtype, tokens, heads, dim, dev)
    v = _heads_arg(new_values, "new_values", dtype, tokens, heads, dim, dev)
    f32 = torch.float32
    cos_ptr, pairs, _ = _matrix(cos, "cos", (f32,), cos.shape[0] if isinstance(cos, torch.Tensor) and cos.dim() else 0,
                                dev)
    positions = 0
    sin_ptr = 0
    if cos is not None:
        positions = cos.shape[0]
        sin_ptr = _arg(sin, "sin", f32, positions * pairs, dev)
        if not cos.is_contiguous() or sin.shape != cos.shape:
            raise ValueError("cos and sin must be contiguous and agree in shape")
        if 2 * pairs > dim:
            raise ValueError("cos and sin have more pairs than a head")
    elif sin is not None:
        raise ValueError("sin needs cos")
    q, q_heads, o = (0, 0, 0), 0, (0, 0, 0)
    if queries is not None:
        q = _heads_arg(queries, "queries", dtype, tokens, None, dim, dev)
        q_heads = queries.shape[1]
        if queries_out is None:
            queries_out = _new((tokens, q_heads, dim), dtype, cache.device, stream)
        o = _heads_arg(queries_out, "queries_out", dtype, tokens, q_heads, dim, dev)
        _distinct(queries_out, "queries_out")
    elif queries_out is not None:
        raise ValueError("queries_out needs queries")
    new = _native.pack_new_tokens(tokens, kind, *k, *v, q[0], q_heads, q[1], q[2], *o, cos_ptr, sin_ptr, positions,
                                  pairs, bool(interleaved))
    _native.check(_native.lib().pages_append(*args, _optional(status, "status", torch.int32, args[3], dev), new, sh),
                  "pages_append")
    return queries_out


def pages_attend(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, queries: torch.Tensor, *,
                 starts: torch.Tensor | None = None, scale: float | None = None, out: torch.Tensor | None = None,
                 stream=None, workspace: Workspace | None = None) -> torch.Tensor:
    """Attention of queries [tokens, q_heads, dim] (float16 or bfloat16) over
    their rows' tokens in a cache of float8_e4m3fn: every token sees those at
    positions up to its own, query head h reads key head h // (q_heads //
    heads). Rows, starts and positions as pages_append; scale multiplies the
    products (None: dim ** -0.5). dim is a multiple of 16 up to 256; a cache's
    addresses and strides are multiples of 16 bytes, and so are the queries'.
    The scales of blocks that hold a seen token must be finite and not below 0
    (as pages_append writes them); other blocks may hold anything. A query that
    sees no token gets zeros. Returns out (a new tensor by default, else one
    that shares no memory with queries; tokens behind the last row's are left
    alone in it)."""
    shape = _tensor(queries, "queries").shape
    tokens = shape[0] if len(shape) else 0
    args = _cache_rows(cache, table, lens, starts, tokens)
    dev, dim = cache.device.index, cache.dim
    sh = _launch_stream(stream, dev)
    if cache.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"the cache must have dtype torch.float8_e4m3fn, got {cache.dtype}")
    dtype = queries.dtype
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise TypeError(f"queries must have dtype torch.float16 or torch.bfloat16, got {dtype}")
    q = _heads_arg(queries, "queries", dtype, tokens, None, dim, dev)
    q_heads = shape[1]
    if cache.heads == 0 or q_heads == 0 or q_heads % cache.heads:
        raise ValueError("queries must have a multiple of the cache's heads")
    if out is None:
        out = _new((tokens, q_heads, dim), dtype, cache.device, stream)
    o = _heads_arg(out, "out", dtype, tokens, q_heads, dim, dev)
    _distinct(out, "out")
    if workspace is None:
        workspace = Workspace.get(_native.OP_ATTEND, tokens, cache.device, sh)
    elif workspace.buf.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev}")
    _native.check(_native.lib().pages_attend(
        *args, tokens, q[0], _LOGIT_TYPES[dtype], q_heads, q[1], q[2], *o, dim**-0.5 if scale is None else scale,
        workspace.ptr, workspace.nbytes, sh), "pages_attend")
    return out


def check(stream=None, workspace: Workspace | None = None, device=None) -> int:
    """Synchronise the stream and raise if a kernel that used the stream's
    cached workspace reported a device-side error (a carry-wait timeout)."""
    sh = _stream_handle(stream)
    if workspace is None:
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        workspace = Workspace._cache.get((dev.index, sh))
        if workspace is None:
            torch.cuda.synchronize()
            return _native.OK
    status = _native.lib().u32scan_check(workspace.ptr, sh)
    _native.check(status, "u32scan_check")
    return status
