"""Stand-ins for CUDA tensors, streams and the native library, so that what
the Python binding does before a launch (which stream, which device, which
refusals) is tested without a GPU. Nothing is launched: the library's calls are
recorded and answer OK."""

import contextlib

import torch

from u32_prefix_scan_gb300 import _native


class Tensor(torch.Tensor):
    """A host tensor that says it lies on cuda:`dev` in memory of `stream`."""

    is_cuda = True
    dev, stream, recorded = 0, None, ()

    @property
    def device(self):
        return torch.device("cuda", self.dev)

    def get_device(self):
        return self.dev

    def record_stream(self, stream):
        self.recorded = (*self.recorded, stream.cuda_stream)


class Stream:
    """A stream by its handle; `pool` numbers those that get one by themselves."""

    pool = 5000

    def __init__(self, handle, dev=0):
        self.cuda_stream, self.device, self.device_index = handle, torch.device("cuda", dev), dev
        self.waited = []

    def wait_stream(self, other):
        self.waited.append(other.cuda_stream)


def external_stream(handle, device=None):
    """As torch's: handle 0 stands for no handle, and gives a stream of the pool."""
    if handle == 0:
        Stream.pool += 1
        handle = Stream.pool
    return Stream(handle, torch.device(device or "cuda:0").index or 0)


class Library:
    """Records the library's calls."""

    def __init__(self, workspace_bytes=4096):
        self.calls = []
        self.workspace_bytes = workspace_bytes

    def u32scan_workspace_bytes(self, op, n):
        return self.workspace_bytes

    def __getattr__(self, name):
        if name not in _native.SIGNATURES:
            raise AttributeError(name)

        def call(*args):
            self.calls.append((name, args))
            return _native.OK

        return call


class Device:
    """A machine with two GPUs, cuda:0 current, and `current` its stream."""

    def __init__(self, monkeypatch):
        from u32_prefix_scan_gb300 import api

        self.lib = Library()
        self.dev = 0
        self.current = Stream(1000)
        self.default = Stream(0)
        self.external = []
        self.workspaces = {}

        def new_external(handle, device=None):
            self.external.append(external_stream(handle, device))
            return self.external[-1]

        @contextlib.contextmanager
        def use(stream):
            was, self.current = self.current, stream
            yield
            self.current = was

        def made(make):
            def f(*args, device=None, **kw):
                if torch.device(device if device is not None else "cpu").type != "cuda":
                    return make(*args, device=device, **kw)
                t = make(*args, **kw).as_subclass(Tensor)
                t.dev, t.stream = torch.device(device).index or 0, self.current.cuda_stream
                return t

            return f

        patch = monkeypatch.setattr
        patch(_native, "lib", lambda: self.lib)
        patch(api, "_raw_stream", lambda dev: self.current.cuda_stream)
        patch(api.Workspace, "_cache", self.workspaces)
        patch(torch, "empty", made(torch.empty))
        patch(torch, "zeros", made(torch.zeros))
        patch(torch, "tensor", made(torch.tensor))
        patch(torch.cuda, "current_device", lambda: self.dev)
        patch(torch.cuda, "current_stream", lambda device=None: self.current)
        patch(torch.cuda, "default_stream", lambda device=None: self.default)
        patch(torch.cuda, "ExternalStream", new_external)
        patch(torch.cuda, "stream", use)

    def new(self, *shape, dtype=torch.int32, dev=0):
        return torch.zeros(*shape, dtype=dtype, device=f"cuda:{dev}")
