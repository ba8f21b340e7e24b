"""GPU parity of adjust_logits against the CPU oracle: bit for bit, whatever
the type, vocabulary, strides, lists and masks."""

import numpy as np
import pytest

import oracle
from u32_prefix_scan_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAMES = ("history", "history_lens", "prompt_lens", "repetition", "presence", "frequency", "bias_tokens", "bias", "allowed")


@pytest.fixture(scope="module")
def u():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from u32_prefix_scan_gb300 import build

    build.build()
    import u32_prefix_scan_gb300 as u

    return u


def rules_for(rows, vocab, seed, width=40, biases=6, mask=True):
    rng = np.random.default_rng(seed)
    r = {
        "history": (rng.random((rows, width)) ** 2 * (vocab + 2)).astype(np.int32) - 1,  # -1 and vocab: skipped
        "history_lens": rng.integers(-2, width + 3, rows).astype(np.int32),
        "prompt_lens": rng.integers(-2, width + 3, rows).astype(np.int32),
        "repetition": rng.choice(np.float32([1.0, 1.3, 0.7, 0.0, -1.0, np.nan, np.inf]), rows),
        "presence": rng.choice(np.float32([0.0, 0.5, -0.3, np.nan]), rows),
        "frequency": rng.choice(np.float32([0.0, 0.1, -0.7, np.inf]), rows),
    }
    if biases:
        r["bias_tokens"] = rng.integers(-1, vocab + 1, (rows, biases)).astype(np.int32)  # twice the same among them
        r["bias"] = rng.choice(np.float32([-100.0, 0.1, 3.0, -np.inf]), (rows, biases))
    if mask:
        words = (vocab + 31) // 32
        r["allowed"] = rng.integers(0, 1 << 32, (rows, words), dtype=np.uint64).astype(np.uint32)
        r["allowed"][rows // 2] = 0  # a row that nothing is left of
    return r


def logits_for(rows, vocab, seed, dtype):
    rng = np.random.default_rng(seed)
    x = (3 * rng.standard_normal((rows, vocab))).astype(np.float32)
    x[rng.random((rows, vocab)) < 0.05] = -np.inf
    x[rng.random((rows, vocab)) < 0.02] = np.nan
    x[rng.random((rows, vocab)) < 0.02] = np.inf
    x[rng.random((rows, vocab)) < 0.02] = -0.0
    x[rng.random((rows, vocab)) < 0.02] = 0.0
    return torch.from_numpy(x).to(TYPES[dtype])


def on_gpu(rules):
    return {k: torch.from_numpy(v.view(np.int32) if v.dtype == np.uint32 else v).cuda() for k, v in rules.items()}


def bits(t):
    return t.cpu().contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16).numpy()


def check(got, logits, rules):
    """Equal bits; a NaN that a rule reached may be any."""
    want, touched = oracle.adjust_logits(logits.float().numpy(), **rules)
    want = torch.from_numpy(want).to(logits.dtype)
    want = torch.where(torch.from_numpy(touched), want, logits)
    same = bits(got) == bits(want)
    both_nan = torch.isnan(got.cpu()).numpy() & torch.isnan(want).numpy() & touched
    assert np.all(same | both_nan), np.argwhere(~(same | both_nan))[:5]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 7), (5, 31), (4, 33), (2, 4096), (3, 4097), (7, 50257), (1, 131075)])
def test_every_rule(u, rows, vocab, dtype):
    logits, rules = logits_for(rows, vocab, vocab, dtype), rules_for(rows, vocab, rows)
    check(u.adjust_logits(logits.cuda(), **on_gpu(rules)), logits, rules)


@pytest.mark.parametrize("name", ["history", "repetition", "presence", "frequency", "bias", "allowed", "none"])
def test_one_rule_alone(u, name):
    logits, rules = logits_for(5, 1003, 1, "bf16"), rules_for(5, 1003, 2)
    keep = {"history": ["history"], "bias": ["bias", "bias_tokens"], "allowed": ["allowed"], "none": []}
    kept = {k: rules[k] for k in keep.get(name, ["history", "history_lens", "prompt_lens", name])}
    check(u.adjust_logits(logits.cuda(), **on_gpu(kept)), logits, kept)


@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 255, 257, 5000, 40001])
def test_history_widths(u, width):
    """Short and long histories, tokens that occur thousands of times, every row at another offset."""
    logits = logits_for(3, 9001, width, "f16")
    rules = rules_for(3, 9001, width, width=width)
    rules["history"][1] = 77
    rules["history_lens"][:] = [width, width - 1, width // 2]
    rules["prompt_lens"][:] = [0, width // 3, width]
    rules["repetition"][:] = 1.1
    rules["presence"][:] = 0.25
    rules["frequency"][:] = 0.01
    check(u.adjust_logits(logits.cuda(), **on_gpu(rules)), logits, rules)


@pytest.mark.parametrize("n", [1, 31, 300, 3001])
def test_many_biases_and_the_same_token_twice(u, n):
    logits = logits_for(2, 5003, n, "f32")
    rules = rules_for(2, 5003, n, biases=n)
    rules["bias_tokens"][1] = np.arange(n) % 3  # the last of each holds
    check(u.adjust_logits(logits.cuda(), **on_gpu(rules)), logits, rules)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("off", [0, 1, 3, 8])
def test_strides_offsets_and_in_place(u, dtype, off):
    rows, vocab = 4, 3001
    logits, rules = logits_for(rows, vocab, off, dtype), rules_for(rows, vocab, off + 5)
    g = on_gpu(rules)
    wide = torch.full((rows, vocab + off + 5), 9.0, dtype=TYPES[dtype], device="cuda")
    view = wide[:, off : off + vocab]
    view.copy_(logits)
    check(u.adjust_logits(view, **g), logits, rules)
    out = torch.full((rows, vocab + 2 * off + 1), 7.0, dtype=TYPES[dtype], device="cuda")
    check(u.adjust_logits(view, out=out[:, off : off + vocab], **g), logits, rules)
    assert torch.all(out[:, :off] == 7) and torch.all(out[:, off + vocab :] == 7)
    # lists with gaps between their rows, one mask for all rows
    wide_h = torch.full((rows, 57), 5, dtype=torch.int32, device="cuda")
    wide_h[:, 3:43] = g["history"]
    g["history"] = wide_h[:, 3:43]
    g["allowed"] = g["allowed"][:1].expand(rows, -1)
    rules["allowed"] = np.repeat(rules["allowed"][:1], rows, 0)
    back = u.adjust_logits(view, out=view, **g)
    assert back is view
    check(view, logits, rules)
    assert torch.all(wide[:, :off] == 9) and torch.all(wide[:, off + vocab :] == 9)


def test_rows_and_vocabularies_of_none(u):
    for shape in ((0, 100), (3, 0), (0, 0)):
        x = torch.empty(shape, device="cuda")
        assert u.adjust_logits(x).shape == shape
    x = torch.ones(2, 5, device="cuda")
    h = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    assert torch.equal(u.adjust_logits(x, history=h, repetition=torch.full((2,), 3.0, device="cuda")), x)


def test_refusals(u):
    x = torch.zeros(4, 100, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(u_error()):  # a part of the logits as the output
        u.adjust_logits(x[:, :50], out=x[:, 10:60])
    with pytest.raises(u_error()):
        u.adjust_logits(x[:3], out=x[1:])
    for kw in (dict(out=torch.zeros(4, 99, device="cuda")), dict(allowed=torch.zeros(4, 3, **i32)),
               dict(bias=torch.zeros(4, 3, device="cuda"), bias_tokens=torch.zeros(4, 4, **i32)),
               dict(bias_tokens=torch.zeros(4, 4, **i32)), dict(history=torch.zeros(3, 4, **i32)),
               dict(history_lens=torch.zeros(3, **i32)), dict(history=torch.zeros(4, 8, **i32)[:, ::2])):
        with pytest.raises(ValueError):
            u.adjust_logits(x, **kw)
    for kw in (dict(out=torch.zeros(4, 100, dtype=torch.float16, device="cuda")),
               dict(history=torch.zeros(4, 4, dtype=torch.int64, device="cuda")),
               dict(repetition=torch.zeros(4, dtype=torch.float64, device="cuda"))):
        with pytest.raises(TypeError):
            u.adjust_logits(x, **kw)


def u_error():
    from u32_prefix_scan_gb300 import _native

    return _native.U32ScanError


def test_another_stream_a_graph_and_then_sampling(u):
    """Captured once, replayed with other logits and lists in the same tensors."""
    rows, vocab = 6, 20011
    logits, rules = logits_for(rows, vocab, 3, "bf16").nan_to_num(0.0, 50.0, -50.0), rules_for(rows, vocab, 4)
    x, g = logits.cuda(), on_gpu(rules)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = u.adjust_logits(x, stream=side, **g)
    torch.cuda.current_stream().wait_stream(side)
    check(out, logits, rules)
    words = torch.from_numpy(inputs.splitmix_u32(3, 0, rows).view(np.int32)).cuda()
    graph = torch.cuda.CUDAGraph()
    u.sample_tokens(u.adjust_logits(x, **g), words)
    with torch.cuda.graph(graph):
        out = u.adjust_logits(x, **g)
        tokens, _ = u.sample_tokens(out, words)
    for seed in (11, 12):
        logits, rules = logits_for(rows, vocab, seed, "bf16").nan_to_num(0.0, 50.0, -50.0), rules_for(rows, vocab, seed)
        x.copy_(logits)
        for k, v in on_gpu(rules).items():
            g[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        check(out, logits, rules)
        want, _ = oracle.sample_tokens(out.float().cpu().numpy(), words.cpu().numpy().view(np.uint32))
        assert np.array_equal(tokens.cpu().numpy(), want) and tokens[rows // 2] == -1


# from 304 blocks of four vectors a thread on: 8192 f32 logits a block, 16384 of 16 bits
@pytest.mark.parametrize("rows,vocab,dtype", [(40, 65537, "f32"), (80, 65543, "bf16"), (77, 65536, "f16"), (304, 8201, "f32")])
@pytest.mark.parametrize("off", [0, 3, 8])
def test_large_batches(u, rows, vocab, dtype, off):
    """Rows at any place within a vector, in place too; more names in one slice than a block keeps, and the same ones
    again; a history longer than a slice."""
    logits = logits_for(rows, vocab, off, dtype)
    rules = rules_for(rows, vocab, off + 1, width=9000 if rows < 50 else 700, biases=700)
    rules["bias_tokens"][1] = 5000 + np.arange(700) % 601
    rules["bias_tokens"][2] = np.random.default_rng(off).permutation(8000)[:700]
    g = on_gpu(rules)
    wide = torch.full((rows, vocab + off + 5), 9.0, dtype=TYPES[dtype], device="cuda")
    view = wide[:, off : off + vocab]
    view.copy_(logits)
    out = torch.full_like(wide, 7.0)
    check(u.adjust_logits(view, out=out[:, off : off + vocab], **g), logits, rules)
    assert torch.all(out[:, :off] == 7) and torch.all(out[:, off + vocab :] == 7)
    u.adjust_logits(view, out=view, **g)
    assert np.array_equal(bits(wide[:, off : off + vocab]), bits(out[:, off : off + vocab]))
    assert torch.all(wide[:, :off] == 9) and torch.all(wide[:, off + vocab :] == 9)


@pytest.mark.parametrize("vocab", [1000, 1003, 70001])
def test_results_between_the_logits(u, vocab):
    """Rows of logits and of results in one tensor, every row's beside each other; over each other they are refused."""
    logits, rules = logits_for(6, vocab, 5, "bf16"), rules_for(6, vocab, 6)
    both = torch.full((6, 2, vocab + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    both[:, 0, :vocab] = logits
    g = on_gpu(rules)
    check(u.adjust_logits(both[:, 0, :vocab], out=both[:, 1, :vocab], **g), logits, rules)
    assert np.array_equal(bits(both[:, 0, :vocab]), bits(logits)) and torch.all(both[:, :, vocab:] == 7)
    flat = both.flatten(1)
    for at in (1, vocab - 1):
        with pytest.raises(u_error()):
            u.adjust_logits(flat[:, :vocab], out=flat[:, at : at + vocab], **g)
