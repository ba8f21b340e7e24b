"""What adjust_logits, KVCache, pages_append and pages_attend do in Python
before a launch, on stand-ins for CUDA tensors and streams (no GPU): which
device and stream they take, and what they refuse."""

import pytest

torch = pytest.importorskip("torch")

import u32_prefix_scan_gb300 as u  # noqa: E402
from fake_device import Device, Stream, Tensor  # noqa: E402
from u32_prefix_scan_gb300 import _native  # noqa: E402

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture
def gpu(monkeypatch):
    return Device(monkeypatch)


def on(t, dev=0):
    t = t.as_subclass(Tensor)
    t.dev = dev
    return t


class Args:
    """The arguments of every call, on one device."""

    def __init__(self, gpu, dev=0, dtype=E4M3):
        self.logits, self.rows4 = gpu.new(4, 64, dtype=F32, dev=dev), gpu.new(4, dev=dev)
        self.each, self.matrix = gpu.new(4, dtype=F32, dev=dev), gpu.new(4, 2, dev=dev)
        self.biases = gpu.new(4, 2, dtype=F32, dev=dev)
        self.keys, self.values = (on(torch.zeros(6, 16, 2, 32, dtype=dtype), dev) for _ in range(2))
        coded = dtype is E4M3
        self.scales = [gpu.new(6, 4, 2, dtype=F32, dev=dev) if coded else None for _ in range(2)]
        self.table, self.lens = gpu.new(4, 3, dev=dev), gpu.new(4, dev=dev)
        self.k, self.v = (gpu.new(4, 2, 32, dtype=BF16, dev=dev) for _ in range(2))
        self.q = gpu.new(4, 6, 32, dtype=BF16, dev=dev)
        self.angles = gpu.new(50, 16, dtype=F32, dev=dev)
        self.cache = u.KVCache(self.keys, self.values, *self.scales)

    def calls(self):
        c = (self.cache, self.table, self.lens)
        return {
            "adjust_logits": lambda **kw: u.adjust_logits(self.logits, history=self.matrix, history_lens=self.rows4,
                                                          repetition=self.each, bias=self.biases,
                                                          bias_tokens=self.matrix, allowed=self.matrix, **kw),
            "pages_append": lambda **kw: u.pages_append(*c, self.k, self.v, cos=self.angles, sin=self.angles,
                                                        queries=self.q, status=self.rows4, **kw),
            "pages_attend": lambda **kw: u.pages_attend(*c, self.q, **kw),
        }


CALLS = ["adjust_logits", "pages_append", "pages_attend"]


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
def test_another_device_is_refused(gpu, name):
    with pytest.raises(ValueError, match="cuda:1.*cuda:0 is current"):
        Args(gpu, 1).calls()[name]()
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        Args(gpu).calls()[name](stream=Stream(77, 1))
    with pytest.raises(ValueError, match="workspace must be on cuda:0"):
        Args(gpu).calls()["pages_attend"](workspace=u.Workspace(4096, torch.device("cuda", 1)))
    assert gpu.lib.calls == []


def test_every_tensor_on_the_cache_or_logits_device(gpu):
    a, b = Args(gpu), Args(gpu, 1)
    c = (a.cache, a.table, a.lens)
    for call in (lambda: u.pages_append(a.cache, b.table, a.lens, a.k, a.v),
                 lambda: u.pages_append(a.cache, a.table, b.lens, a.k, a.v),
                 lambda: u.pages_append(*c, b.k, a.v), lambda: u.pages_append(*c, a.k, b.v),
                 lambda: u.pages_append(*c, a.k, a.v, starts=gpu.new(5, dev=1)),
                 lambda: u.pages_append(*c, a.k, a.v, status=b.rows4),
                 lambda: u.pages_append(*c, a.k, a.v, cos=b.angles, sin=a.angles),
                 lambda: u.pages_append(*c, a.k, a.v, cos=a.angles, sin=b.angles),
                 lambda: u.pages_append(*c, a.k, a.v, queries=b.q),
                 lambda: u.pages_append(*c, a.k, a.v, queries=a.q, queries_out=b.q),
                 lambda: u.pages_attend(*c, b.q), lambda: u.pages_attend(*c, a.q, out=b.q),
                 lambda: u.adjust_logits(a.logits, history=b.matrix),
                 lambda: u.adjust_logits(a.logits, presence=b.each),
                 lambda: u.adjust_logits(a.logits, out=b.logits)):
        with pytest.raises(ValueError, match="must be on cuda:0"):
            call()
    for kw in (dict(keys=b.keys), dict(values=b.values), dict(key_scales=b.scales[0]), dict(value_scales=b.scales[1])):
        args = dict(keys=a.keys, values=a.values, key_scales=a.scales[0], value_scales=a.scales[1]) | kw
        with pytest.raises(ValueError):
            u.KVCache(**args)
    assert gpu.lib.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_outputs_lie_in_memory_of_the_stream_that_writes_them(gpu, name):
    out = Args(gpu).calls()[name](stream=Stream(77))
    assert (out.stream, out.recorded) == (77, (1000,))
    out = Args(gpu).calls()[name]()
    assert (out.stream, out.recorded) == (1000, ())


@pytest.mark.parametrize("other", [None, 3, [1, 2], "words"])
def test_arguments_that_are_no_tensors(gpu, other):
    a = Args(gpu)
    c = (a.cache, a.table, a.lens)
    calls = {
        "logits": lambda: u.adjust_logits(other),
        "keys": lambda: u.KVCache(other, a.values, *a.scales),
        "values": lambda: u.KVCache(a.keys, other, *a.scales),
        "cache": lambda: u.pages_attend(other, a.table, a.lens, a.q),
        "table": lambda: u.pages_attend(a.cache, other, a.lens, a.q),
        "lens": lambda: u.pages_append(a.cache, a.table, other, a.k, a.v),
        "new_keys": lambda: u.pages_append(*c, other, a.v),
        "new_values": lambda: u.pages_append(*c, a.k, other),
        "queries": lambda: u.pages_attend(*c, other),
        "sin": lambda: u.pages_append(*c, a.k, a.v, cos=a.angles, sin=other),
        "bias_tokens": lambda: u.adjust_logits(a.logits, bias=a.biases, bias_tokens=other),
    }
    if other is not None:
        calls |= {name: lambda name=name: u.adjust_logits(a.logits, **{name: other}) for name in (
            "history", "history_lens", "prompt_lens", "repetition", "presence", "frequency", "bias", "allowed", "out")}
        calls |= {name: lambda name=name: u.pages_append(*c, a.k, a.v, **{name: other}) for name in (
            "starts", "status", "cos", "queries")}
        calls["queries_out"] = lambda: u.pages_append(*c, a.k, a.v, queries=a.q, queries_out=other)
        calls["key_scales"] = lambda: u.KVCache(a.keys, a.values, other, a.scales[1])
        calls["value_scales"] = lambda: u.KVCache(a.keys, a.values, a.scales[0], other)
    for name, call in calls.items():
        with pytest.raises(TypeError, match=f"{name} must be a"):
            call()
    assert gpu.lib.calls == []


def test_shapes_types_and_layouts_that_are_refused(gpu):
    a = Args(gpu)
    c = (a.cache, a.table, a.lens)
    new = gpu.new
    wide = new(4, 2, 64, dtype=BF16)
    for call in (
            lambda: u.KVCache(a.keys, on(a.values[:, :, :1]), *a.scales),
            lambda: u.KVCache(on(a.keys[0]), on(a.values[0]), *a.scales),
            lambda: u.KVCache(on(a.keys[:, :0]), on(a.values[:, :0]), *a.scales),
            lambda: u.KVCache(on(a.keys[:, :, :, :0]), on(a.values[:, :, :, :0]), *a.scales),
            lambda: u.KVCache(a.keys, a.values), lambda: u.KVCache(a.keys, a.values, a.scales[0]),
            lambda: u.KVCache(a.keys, a.values, new(6, 3, 2, dtype=F32), new(6, 3, 2, dtype=F32)),
            lambda: u.KVCache(a.keys, a.values, new(6, 0, 2, dtype=F32), new(6, 0, 2, dtype=F32)),
            lambda: u.KVCache(a.keys, a.values, a.scales[0], new(6, 2, 2, dtype=F32)),
            lambda: u.KVCache(a.keys, a.values, new(6, 4, 3, dtype=F32), new(6, 4, 3, dtype=F32)),
            lambda: u.KVCache(on(a.keys.transpose(2, 3)), on(a.values.transpose(2, 3)), *a.scales),
            lambda: u.KVCache(on(a.keys[:1].expand(6, -1, -1, -1)), on(a.values[:1].expand(6, -1, -1, -1)), *a.scales),
            lambda: u.KVCache(a.keys, a.values, *[on(s[:1].expand(6, -1, -1)) for s in a.scales]),
            lambda: u.KVCache(a.keys, a.values, *[on(s.transpose(1, 2).contiguous().transpose(1, 2)) for s in a.scales]),
            lambda: u.pages_append(*c, wide, a.v), lambda: u.pages_append(*c, a.k, on(a.v[:3])),
            lambda: u.pages_append(*c, on(wide[:, :, ::2]), a.v), lambda: u.pages_append(*c, on(a.k[:3]), on(a.v[:3])),
            lambda: u.pages_append(*c, a.k, a.v, starts=new(4)), lambda: u.pages_append(*c, a.k, a.v, sin=a.angles),
            lambda: u.pages_append(*c, a.k, a.v, cos=a.angles, sin=new(50, 15, dtype=F32)),
            lambda: u.pages_append(*c, a.k, a.v, cos=new(50, 17, dtype=F32), sin=new(50, 17, dtype=F32)),
            lambda: u.pages_append(*c, a.k, a.v, queries_out=a.q),
            lambda: u.pages_append(*c, a.k, a.v, queries=a.q, queries_out=on(a.q[:1].expand(4, -1, -1))),
            lambda: u.pages_append(*c, a.k, a.v, status=new(3)),
            lambda: u.pages_append(a.cache, on(a.table[:1].expand(4, -1)), a.lens, a.k, a.v),
            lambda: u.pages_append(a.cache, a.table, new(5), a.k, a.v),
            lambda: u.pages_attend(*c, on(a.q[:, :5])), lambda: u.pages_attend(*c, on(a.q[:, :0])),
            lambda: u.pages_attend(*c, a.q, out=on(a.q[:, :4])),
            lambda: u.pages_attend(*c, a.q, out=on(a.q[:, :1].expand(-1, 6, -1))),
    ):
        with pytest.raises(ValueError):
            call()
    f32, f64 = new(4, 2, 32, dtype=F32), torch.float64
    plain = Args(gpu, dtype=BF16)
    for call in (lambda: u.KVCache(on(a.keys.view(torch.uint8)), a.values, *a.scales),
                 lambda: u.KVCache(a.keys, a.values, *[s.to(f64) for s in a.scales]),
                 lambda: u.pages_append(*c, a.k, f32), lambda: u.pages_append(*c, new(4, 2, 32), a.v),
                 lambda: u.pages_append(plain.cache, a.table, a.lens, f32, f32),
                 lambda: u.pages_attend(plain.cache, a.table, a.lens, a.q),
                 lambda: u.pages_attend(*c, new(4, 6, 32, dtype=F32)),
                 lambda: u.pages_attend(*c, a.q, out=new(4, 6, 32, dtype=torch.float16)),
                 lambda: u.pages_attend(a.cache, a.table.long(), a.lens, a.q)):
        with pytest.raises(TypeError):
            call()
    assert gpu.lib.calls == []


def test_what_the_library_gets(gpu):
    """Strides in elements; those of sizes of one are none."""
    a = Args(gpu)
    u.pages_attend(a.cache, a.table, a.lens, a.q, starts=gpu.new(5), scale=0.5)
    args = gpu.lib.calls[-1][1]
    assert args[2:5] == (3, 4, 3) and args[7] == 4 and args[9:13] == (_native.BF16, 6, 192, 32) and args[16] == 0.5
    s = a.cache.struct
    assert (s.type, s.pages, s.page_tokens, s.heads, s.dim) == (_native.E4M3, 6, 16, 2, 32)
    assert (s.page_stride, s.token_stride, s.head_stride, s.blocks, s.scale_stride) == (1024, 64, 32, 4, 8)
    u.pages_append(a.cache, a.table, a.lens, a.k, a.v, cos=a.angles, sin=a.angles, interleaved=True)
    n = _native.NewTokensStruct.from_buffer_copy(gpu.lib.calls[-1][1][8])
    assert (n.tokens, n.type, n.key_token_stride, n.key_head_stride, n.positions, n.pairs) == (4, _native.BF16, 64, 32, 50, 16)
    assert n.queries is None and n.interleaved == 1
    u.adjust_logits(a.logits, allowed=on(a.matrix[:1].expand(4, -1)))
    r = _native.LogitRulesStruct.from_buffer_copy(gpu.lib.calls[-1][1][7])
    assert r.history is None and r.allowed_stride == 0 and r.allowed == a.matrix.data_ptr()


def test_packed_arguments_are_the_structures():
    for kind, pack in ((_native.LogitRulesStruct, _native.pack_logit_rules), (_native.NewTokensStruct, _native.pack_new_tokens)):
        values = [i + 1 for i in range(len(kind._fields_))]
        assert pack(*values) == bytes(kind(*values))


def test_a_cache_that_shares_memory_is_only_read(gpu):
    """Keys that are the values, or a part of them; scales likewise. Views of one page beside each other are not."""
    a = Args(gpu)
    room = on(torch.zeros(6, 3, 16, 2, 32, dtype=E4M3))
    page = on(torch.zeros(6, 4, 16, 2, 40, dtype=E4M3))
    scales = gpu.new(6, 9, 2, dtype=F32)

    def views(t, i, j):
        return on(t[:, i]), on(t[:, j])

    shared = [(a.keys, a.keys, *a.scales), (on(room[:, 0]), on(room[:, 0]), *a.scales),
              (on(room.flatten(1, 2)[:, :16]), on(room.flatten(1, 2)[:, 15:31]), *a.scales),
              (on(room.flatten(1, 2)[:, 5:21]), on(room.flatten(1, 2)[:, :16]), *a.scales),
              (on(page[:, 0, :, :, :32]), on(page[:, 0, :, :, 8:]), *a.scales),
              (a.keys, a.values, a.scales[0], a.scales[0]),
              (a.keys, a.values, on(scales[:, :4]), on(scales[:, 3:7])),
              (a.keys, a.values, on(scales[:, 5:]), on(scales[:, 4:8]))]
    apart = [(a.keys, a.values, *a.scales), (*views(room, 0, 1), *a.scales), (*views(room, 2, 0), *a.scales),
             (*views(page, 3, 1), *a.scales), (a.keys, a.values, on(scales[:, :4]), on(scales[:, 4:8])),
             (on(room[:1, 0]), on(room[1:2, 0]), on(a.scales[0][:1]), on(a.scales[0][1:2])),
             (on(page[..., :8]).flatten(1, 2)[:, :16], on(page[..., 8:16]).flatten(1, 2)[:, :16], *a.scales)]
    none = [on(torch.zeros(0, 16, 2, 32, dtype=E4M3)) for _ in range(2)]
    apart.append((*none, *[on(torch.zeros(0, 4, 2)) for _ in range(2)]))
    rows = (a.table, a.lens)
    for parts in shared:
        cache = u.KVCache(*map(on, parts))
        with pytest.raises(ValueError, match="share memory"):
            u.pages_append(cache, *rows, a.k, a.v)
        u.pages_attend(cache, *rows, on(a.q))
    reads = len(gpu.lib.calls)
    for parts in apart:
        cache = u.KVCache(*map(on, parts))
        k = gpu.new(4, 2, cache.dim, dtype=BF16)
        u.pages_append(cache, *rows, k, k)
    assert reads == len(shared) and len(gpu.lib.calls) == reads + len(apart)
