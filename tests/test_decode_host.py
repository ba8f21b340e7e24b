"""What the decode step's Python calls do before a launch, on stand-ins for
CUDA tensors and streams (no GPU): which device and stream they take, and
what they refuse."""

import pytest

torch = pytest.importorskip("torch")

import u32_prefix_scan_gb300 as u  # noqa: E402
from fake_device import Device, Stream  # noqa: E402


@pytest.fixture
def gpu(monkeypatch):
    return Device(monkeypatch)


class Args:
    """The arguments of every call, on one device."""

    def __init__(self, gpu, dev=0):
        self.logits, self.words = gpu.new(4, 8, dtype=torch.float32, dev=dev), gpu.new(4, dev=dev)
        self.table, self.lens, self.refs = gpu.new(4, 8, dev=dev), gpu.new(4, dev=dev), gpu.new(50, dev=dev)
        self.pool = object.__new__(u.PagePool)
        self.pool.device, self.pool.struct, self.pool.pages = torch.device("cuda", dev), None, 50

    def calls(self):
        cache = (self.table, self.lens, self.refs, 16)
        return {
            "sample_tokens": lambda **kw: u.sample_tokens(self.logits, self.words, **kw),
            "pages_copy": lambda **kw: u.pages_copy(self.pool, self.lens, self.lens, **kw),
            "pages_fork": lambda **kw: u.pages_fork(*cache, parent=self.lens, grow=self.lens, pool=self.pool, **kw),
            "pages_free": lambda **kw: u.pages_free(*cache, self.lens, **kw),
            "pages_compact": lambda **kw: u.pages_compact(self.pool, *cache, **kw),
        }


CALLS = ["sample_tokens", "pages_copy", "pages_fork", "pages_free", "pages_compact"]


@pytest.mark.parametrize("name", CALLS)
def test_calls_take_the_current_device_and_stream(gpu, name):
    Args(gpu).calls()[name]()
    assert [c[0] for c in gpu.lib.calls] == [name] and gpu.lib.calls[0][1][-1] == 1000
    Args(gpu).calls()[name](stream=Stream(77))
    assert gpu.lib.calls[1][1][-1] == 77
    gpu.dev, gpu.current = 1, Stream(2000, 1)
    Args(gpu, 1).calls()[name]()
    assert gpu.lib.calls[2][1][-1] == 2000


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(gpu, name):
    """The library launches on the current device: another's pointers would
    fault there."""
    with pytest.raises(ValueError, match="cuda:1.*cuda:0 is current"):
        Args(gpu, 1).calls()[name]()
    with pytest.raises(ValueError, match="cuda:1.*cuda:0 is current"):
        Args(gpu, 1).calls()[name](stream=Stream(77, 1))
    assert gpu.lib.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(gpu, name):
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        Args(gpu).calls()[name](stream=Stream(77, 1))
    assert gpu.lib.calls == []


@pytest.mark.parametrize("name", ["pages_fork", "pages_free", "pages_compact"])
def test_a_workspace_of_another_device_is_refused(gpu, name):
    Args(gpu).calls()[name](workspace=u.Workspace(4096, torch.device("cuda", 0)))
    with pytest.raises(ValueError, match="workspace must be on cuda:0"):
        Args(gpu).calls()[name](workspace=u.Workspace(4096, torch.device("cuda", 1)))
    assert len(gpu.lib.calls) == 1


def cleared_workspace(gpu, stream):
    """The workspace that a first call on `stream` gets; it is filled on the current one."""
    a = Args(gpu)
    u.pages_free(a.table, a.lens, a.refs, 16, a.lens, stream=stream)
    (ws,) = gpu.workspaces.values()
    assert ws.buf.stream == gpu.current.cuda_stream == 1000
    return ws


def test_a_workspace_is_filled_before_another_stream_uses_it(gpu):
    ws = cleared_workspace(gpu, Stream(77))
    (other,) = gpu.external
    assert (other.cuda_stream, other.waited, ws.buf.recorded) == (77, [1000], (77,))


def test_a_workspace_is_filled_before_the_default_stream_uses_it(gpu):
    """Handle 0 names the default stream, and no other waits in its place."""
    ws = cleared_workspace(gpu, gpu.default)
    assert (gpu.default.waited, ws.buf.recorded) == ([1000], (0,))


def test_a_workspace_of_the_current_stream_waits_for_nothing(gpu):
    ws = cleared_workspace(gpu, None)
    assert (gpu.external, gpu.default.waited, ws.buf.recorded) == ([], [], ())


@pytest.mark.parametrize("name", ["sample_tokens", "pages_fork", "pages_free", "pages_compact"])
def test_outputs_lie_in_memory_of_the_stream_that_writes_them(gpu, name):
    """Memory that the current stream gave back may still be in use there when
    another stream writes to it; and the outputs may still be in use on the
    current stream when they are given back."""
    outs = Args(gpu).calls()[name](stream=Stream(77))
    for out in [outs] if isinstance(outs, torch.Tensor) else outs:
        assert (out.stream, out.recorded) == (77, (1000,))
    outs = Args(gpu).calls()[name](stream=gpu.default)
    for out in [outs] if isinstance(outs, torch.Tensor) else outs:
        assert (out.stream, out.recorded) == (0, (1000,))
    for kw in ({}, dict(stream=gpu.current)):
        outs = Args(gpu).calls()[name](**kw)
        for out in [outs] if isinstance(outs, torch.Tensor) else outs:
            assert (out.stream, out.recorded) == (1000, ())


@pytest.mark.parametrize("other", [None, 3, [1, 2, 3, 4], "words"])
def test_arguments_that_are_no_tensors(gpu, other):
    """A TypeError that names the argument, whichever it is."""
    a = Args(gpu)
    cache = (a.table, a.lens, a.refs, 16)
    calls = {
        "logits": lambda: u.sample_tokens(other, a.words),
        "random": lambda: u.sample_tokens(a.logits, other),
        "src": lambda: u.pages_copy(a.pool, other, a.lens),
        "dst": lambda: u.pages_copy(a.pool, a.lens, other),
        "pool": lambda: u.pages_copy(other, a.lens, a.lens),
        "table": lambda: u.pages_free(other, a.lens, a.refs, 16, a.lens),
        "lens": lambda: u.pages_free(a.table, other, a.refs, 16, a.lens),
        "refs": lambda: u.pages_free(a.table, a.lens, other, 16, a.lens),
        "release": lambda: u.pages_free(*cache, other),
    }
    if other is not None:  # may be left out
        calls |= {
            "temperature": lambda: u.sample_tokens(a.logits, a.words, temperature=other),
            "top_k": lambda: u.sample_tokens(a.logits, a.words, top_k=other),
            "top_p": lambda: u.sample_tokens(a.logits, a.words, top_p=other),
            "min_p": lambda: u.sample_tokens(a.logits, a.words, min_p=other),
            "tokens": lambda: u.sample_tokens(a.logits, a.words, tokens=other),
            "probs": lambda: u.sample_tokens(a.logits, a.words, probs=other),
            "count": lambda: u.pages_copy(a.pool, a.lens, a.lens, other),
            "parent": lambda: u.pages_fork(*cache, parent=other),
            "grow": lambda: u.pages_fork(*cache, grow=other),
            "status": lambda: u.pages_fork(*cache, status=other),
            "free_pages": lambda: u.pages_fork(*cache, free_pages=other),
            "freed": lambda: u.pages_free(*cache, a.lens, freed=other),
            "live": lambda: u.pages_compact(a.pool, *cache, live=other),
            "remap": lambda: u.pages_compact(a.pool, *cache, remap=other),
        }
    for name, call in calls.items():
        with pytest.raises(TypeError, match=f"{name} must be a"):
            call()
    assert gpu.lib.calls == []


def test_workspace_sizes_are_those_of_the_loaded_library(gpu, monkeypatch):
    """Another library (other launch shapes, swapped in by tests) may need more
    for the same operation and size."""
    from fake_device import Library
    from u32_prefix_scan_gb300 import api

    args = (u._native.OP_PAGES, 12345, torch.device("cuda", 0), 1000)
    assert api.Workspace.get(*args).nbytes == 4096
    first, gpu.lib = gpu.lib, Library(workspace_bytes=8192)
    assert api.Workspace.get(*args).nbytes == 8192
    gpu.workspaces.clear()
    gpu.lib = first
    assert api.Workspace.get(*args).nbytes == 4096
