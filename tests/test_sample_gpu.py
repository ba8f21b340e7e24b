"""GPU parity of sample_tokens against the CPU oracle: tokens and
probabilities are equal bit for bit, whatever the type, vocabulary, stride,
filters and shape of the distribution (peaked, flat, tied, sorted, masked,
with infinities and NaN)."""

import numpy as np
import pytest

import oracle
from u32_prefix_scan_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def u():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from u32_prefix_scan_gb300 import build

    build.build()
    import u32_prefix_scan_gb300 as u

    return u


def logits_for(kind, rows, n, seed):
    rng = np.random.default_rng(seed)
    x = 2.5 * rng.standard_normal((rows, n))
    if kind == "peaked":
        x[np.arange(rows)[:, None], rng.integers(0, n, (rows, 12))] += rng.uniform(4, 14, (rows, 12))
    elif kind == "flat":  # every token counts: wide nuclei, huge sums
        x *= 0.02
    elif kind == "equal":
        x[:] = 1.25
    elif kind == "tied":  # few distinct values, long ties at every cut
        x = np.round(x)
    elif kind == "up":
        x.sort(axis=1)
    elif kind == "down":
        x = -np.sort(-x, axis=1)
    elif kind == "far":  # one token takes everything, the rest lie past the weights' range
        x[:, n // 2] = 300.0
    elif kind == "masked":
        x[rng.random((rows, n)) < 0.97] = -np.inf
        x[0] = -np.inf
        if n > 3:
            x[rows // 2, 1:] = np.nan
            x[-1, n - 1] = np.nan
    elif kind == "wide":  # spread over every exponent, both signs and zeros
        x = np.sign(x) * np.exp2(rng.uniform(-40, 15, (rows, n)))
        x[rng.random((rows, n)) < 0.1] = 0.0
        x[rng.random((rows, n)) < 0.1] = -0.0
    elif kind == "inf":
        x[:, n // 3] = np.inf
        x[:, n - 1] = np.inf
    elif kind == "lowest":  # masked with the type's lowest value
        x[:, n // 2 :] = -65504.0
    return x.astype(np.float32)


def params_for(mode, rows, seed):
    rng = np.random.default_rng(seed + 1000)
    pick = lambda v, t: rng.choice(np.array(v, dtype=t), rows)  # noqa: E731
    if mode == "plain":
        return {}
    if mode == "greedy":
        return dict(temperature=pick([0.0, -1.0, np.nan], np.float32))
    if mode == "top_k":
        return dict(temperature=pick([0.6, 1.0], np.float32), top_k=pick([1, 2, 7, 50, 300, 3000], np.int32))
    if mode == "top_p":
        return dict(top_p=pick([1e-7, 0.3, 0.9, 0.999, 0.9999999], np.float32))
    if mode == "min_p":
        return dict(temperature=pick([0.7, 1.4], np.float32), min_p=pick([1e-9, 0.01, 0.2, 1.0, 3.0], np.float32))
    if mode == "off":  # values that switch a filter off
        return dict(temperature=pick([1.0, np.inf, 1e-30, 1e30], np.float32), top_k=pick([0, -5, 2**31 - 1], np.int32),
                    top_p=pick([0.0, 1.0, 2.0, -1.0, np.nan], np.float32), min_p=pick([0.0, -1.0, np.nan], np.float32))
    return dict(temperature=pick([0.0, 0.5, 1.0, 3.0], np.float32), top_k=pick([0, 1, 20, 64, 500], np.int32),
                top_p=pick([1.0, 0.5, 0.9, 0.99], np.float32), min_p=pick([0.0, 0.0, 0.05], np.float32))


def as_type(x, dtype):
    """The device tensor and the values it holds, as float32."""
    t = torch.from_numpy(x).to(TYPES[dtype])
    return t.cuda(), t.float().numpy()


def run(u, dev, words, params, **kw):
    p = {k: torch.from_numpy(v).cuda() for k, v in params.items()}
    r = torch.from_numpy(words.view(np.int32).copy()).cuda()
    tok, prob = u.sample_tokens(dev, r, **p, **kw)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), prob.cpu().numpy()


def check(u, x, dtype, words, params):
    dev, held = as_type(x, dtype)
    got = run(u, dev, words, params)
    want = oracle.sample_tokens(held, words, **params)
    assert np.array_equal(got[0], want[0])
    assert np.array_equal(got[1].view(np.uint32), want[1].view(np.uint32))


KINDS = ["peaked", "flat", "equal", "tied", "up", "down", "far", "masked", "wide", "inf", "lowest"]
MODES = ["plain", "greedy", "top_k", "top_p", "min_p", "off", "mixed"]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("kind", KINDS)
def test_sample_matches_the_oracle(u, kind, mode, dtype):
    for n, rows in ((13, 9), (1000, 6), (5003, 5), (40001, 3)):
        seed = n + 7 * KINDS.index(kind) + MODES.index(mode)
        check(u, logits_for(kind, rows, n, seed), dtype, inputs.splitmix_u32(11, 0, rows, start=seed),
              params_for(mode, rows, seed))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 31, 32, 33, 255, 1023, 1025, 4096, 8191, 8193, 16385, 32769, 65537, 98305,
                               131072, 200003, 262144, 262145, 524289])
def test_vocabulary_sizes(u, n, dtype):
    rows = 3
    for mode in ("plain", "mixed", "top_p"):
        check(u, logits_for("peaked", rows, n, n), dtype, inputs.splitmix_u32(12, 0, rows, start=n),
              params_for(mode, rows, n))


@pytest.mark.parametrize("kind", ["peaked", "flat", "equal", "tied"])
def test_largest_vocabulary(u, kind):
    n = 1 << 22
    for mode in ("plain", "mixed"):
        check(u, logits_for(kind, 2, n, 5), "bf16", inputs.splitmix_u32(13, 0, 2), params_for(mode, 2, 5))


@pytest.mark.parametrize("rows", [1, 2, 17, 151, 153, 700])
def test_row_counts(u, rows):
    n = 2000
    check(u, logits_for("peaked", rows, n, rows), "f32", inputs.splitmix_u32(14, 0, rows),
          params_for("mixed", rows, rows))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
@pytest.mark.parametrize("stride", [1003, 1004, 1011, 0])
def test_strides_and_alignment(u, dtype, offset, stride):
    rows, n = 6, 1003
    x = logits_for("peaked", 8, 1024, 3).reshape(-1)
    dev, held = as_type(x, dtype)
    view = torch.as_strided(dev, (rows, n), (stride, 1), offset)
    rowsv = np.stack([held[offset + b * stride :][:n] for b in range(rows)])
    words, params = inputs.splitmix_u32(15, 0, rows), params_for("mixed", rows, offset)
    got = run(u, view, words, params)
    want = oracle.sample_tokens(rowsv, words, **params)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert np.array_equal(dev.float().cpu().numpy(), held)  # only read


@pytest.mark.parametrize("n", [50257, 131072])
def test_ends_of_the_word_range(u, n):
    """The lowest and the highest word: the first and the last kept token."""
    x = logits_for("peaked", 4, n, 8)
    words = np.array([0, 0xFFFFFFFF, 1 << 31, 1], dtype=np.uint32)
    for mode in ("plain", "top_k", "top_p"):
        check(u, x, "f32", words, params_for(mode, 4, 8))


def test_a_row_does_not_depend_on_its_batch(u):
    n, rows = 30011, 40
    x = logits_for("peaked", rows, n, 21)
    words, params = inputs.splitmix_u32(16, 0, rows), params_for("mixed", rows, 21)
    dev, _ = as_type(x, "bf16")
    all_tok, all_prob = run(u, dev, words, params)
    for b in (0, 3, 39):
        tok, prob = run(u, dev[b : b + 1], words[b : b + 1], {k: v[b : b + 1] for k, v in params.items()})
        assert tok[0] == all_tok[b] and prob[0] == all_prob[b]


def test_no_rows_and_no_vocabulary(u):
    tok, prob = run(u, torch.empty(0, 100, device="cuda"), np.empty(0, np.uint32), {})
    assert tok.size == 0 and prob.size == 0
    tok, prob = run(u, torch.empty(3, 0, device="cuda"), np.zeros(3, np.uint32), {})
    assert tok.tolist() == [-1] * 3 and prob.tolist() == [0.0] * 3


def test_outputs_stay_inside(u):
    rows, n = 5, 3001
    tokens = torch.full((rows + 4,), 77, dtype=torch.int32, device="cuda")
    probs = torch.full((rows + 4,), 5.0, device="cuda")
    dev, _ = as_type(logits_for("peaked", rows, n, 2), "f32")
    run(u, dev, inputs.splitmix_u32(17, 0, rows), {}, tokens=tokens, probs=probs)
    assert tokens[rows:].tolist() == [77] * 4 and probs[rows:].tolist() == [5.0] * 4


def test_null_arguments_through_the_abi(u):
    from u32_prefix_scan_gb300 import _native

    rows, n = 4, 5000
    dev, held = as_type(logits_for("peaked", rows, n, 4), "bf16")
    words = inputs.splitmix_u32(18, 0, rows)
    r = torch.from_numpy(words.view(np.int32).copy()).cuda()
    tokens = torch.empty(rows, dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert _native.lib().sample_tokens(dev.data_ptr(), _native.BF16, rows, n, n, None, None, None, None, r.data_ptr(),
                                       tokens.data_ptr(), None, st) == _native.OK
    assert np.array_equal(tokens.cpu().numpy(), oracle.sample_tokens(held, words)[0])


@pytest.mark.parametrize("n", [4000, 131072])
def test_other_stream_and_graph(u, n):
    rows = 3
    x = logits_for("peaked", rows, n, 6)
    dev, held = as_type(x, "bf16")
    words, params = inputs.splitmix_u32(19, 0, rows), params_for("mixed", rows, 6)
    want = oracle.sample_tokens(held, words, **params)
    p = {k: torch.from_numpy(v).cuda() for k, v in params.items()}
    r = torch.from_numpy(words.view(np.int32).copy()).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tok, prob = u.sample_tokens(dev, r, **p, stream=side)
    side.synchronize()
    assert np.array_equal(tok.cpu().numpy(), want[0])
    tok.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        u.sample_tokens(dev, r, **p, tokens=tok, probs=prob)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(tok.cpu().numpy(), want[0]) and np.array_equal(prob.cpu().numpy(), want[1])
    r.fill_(0)  # new words are read at every replay
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(tok.cpu().numpy(), oracle.sample_tokens(held, np.zeros(rows, np.uint32), **params)[0])


def test_refusals(u):
    x = torch.zeros(4, 8, device="cuda")
    r = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="dtype"):
        u.sample_tokens(x.double(), r)
    with pytest.raises(ValueError, match="two dimensions"):
        u.sample_tokens(x[0], r)
    with pytest.raises(ValueError, match="adjacent"):
        u.sample_tokens(x.t(), r)
    with pytest.raises(ValueError, match="at least 4"):
        u.sample_tokens(x, r[:3])
    with pytest.raises(TypeError, match="temperature"):
        u.sample_tokens(x, r, temperature=r)
    with pytest.raises(TypeError, match="top_k"):
        u.sample_tokens(x, r, top_k=x[0])
    with pytest.raises(TypeError, match="tokens"):
        u.sample_tokens(x, r, tokens=torch.zeros(4, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("kind", ["peaked", "flat", "equal", "tied", "up", "wide"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_rows_of_every_shape(u, kind, dtype):
    """Rows too long or too even for the lists: the selections within a bin."""
    n, rows = 300007, 3
    x = logits_for(kind, rows, n, 31)
    words = inputs.splitmix_u32(20, 0, rows)
    f, i = np.float32, np.int32
    for params in (dict(top_p=np.array([0.2, 0.9, 0.9999], f)),
                   dict(top_k=np.array([1500, 2047, 200000], i)),
                   dict(top_k=np.array([2049, 60000, 299999], i), top_p=np.array([0.5, 0.97, 0.999], f)),
                   dict(top_k=np.array([5000, 0, 1000], i), top_p=np.array([0.9] * 3, f),
                        min_p=np.array([0.3, 0.01, 1e-6], f)),
                   dict(temperature=np.array([1e4, 0.01, 50.0], f), top_k=np.array([3000, 40, 0], i),
                        top_p=np.array([0.7] * 3, f))):
        check(u, x, dtype, words, params)


def test_largest_f32_vocabulary(u):
    n = 1 << 22
    x = logits_for("peaked", 2, n, 33)
    words = inputs.splitmix_u32(21, 0, 2)
    check(u, x, "f32", words, dict(top_p=np.array([0.9, 1.0], np.float32), top_k=np.array([0, 700], np.int32)))
    check(u, x, "f32", np.array([0xFFFFFFFF, 0], np.uint32), {})


@pytest.fixture(scope="module")
def one_block(u):
    """The library with one block a row: long slices, most of them read again."""
    from u32_prefix_scan_gb300 import _native, build

    return _native.load(build.build_variant("sample_one_block", ["-DU32SCAN_SAMPLE_BLOCKS=1"]))


@pytest.mark.parametrize("kind", ["peaked", "flat", "tied", "masked", "inf"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_any_number_of_blocks_gives_the_same_bits(u, one_block, monkeypatch, kind, dtype):
    from u32_prefix_scan_gb300 import _native

    for n, rows in ((257, 5), (40001, 7), (600011, 2)):
        dev, _ = as_type(logits_for(kind, rows, n, n), dtype)
        for mode in ("plain", "mixed", "top_p", "top_k", "greedy"):
            words, params = inputs.splitmix_u32(22, 0, rows, start=n), params_for(mode, rows, n)
            want = run(u, dev, words, params)
            with monkeypatch.context() as m:
                m.setattr(_native, "_lib", one_block)
                got = run(u, dev, words, params)
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_probabilities_against_softmax_in_64_bits(u, dtype):
    """Without filters the probability is the softmax of the logits held: the
    weight is off by the roundings of its exponent (1.5 ulp of at most 2^-19,
    times ln 2), the polynomial (2e-7) and its floor (2^-31 of the largest),
    the sum by as much, the result by its rounding to float."""
    n, rows = 20011, 64
    dev, held = as_type(logits_for("peaked", rows, n, 41), dtype)
    t = np.linspace(0.4, 3.0, rows).astype(np.float32)
    tok, prob = run(u, dev, inputs.splitmix_u32(23, 0, rows), dict(temperature=t))
    z = held.astype(np.float64) / t[:, None]
    w = np.exp(z - z.max(1, keepdims=True))
    p = (w / w.sum(1, keepdims=True))[np.arange(rows), tok]
    rel = 2 * (1.5 * 2.0**-19 * np.log(2.0) + 2e-7) + n * 2.0**-31 + 2.0**-24
    assert np.all(np.abs(prob - p) <= p * rel + 2.0**-31)


@pytest.mark.parametrize("n", [40, 3000, 70001])
def test_every_size_of_top_p_and_min_p(u, n):
    """The targets ceil(top_p * sum) and ceil(min_p * 2^31) are taken as from
    doubles, from the least float to the last below one."""
    p = [2.0**-149, 2.0**-126, 3 * 2.0**-130, 1e-30, 2.0**-53, 2.0**-24, 2.0**-22, 0.25, 0.5, 1 / 3, 0.1, 0.7, 0.9,
         1 - 2.0**-23, 1 - 2.0**-24]
    p = np.array(p + list(np.random.default_rng(n).random(49)), dtype=np.float32)
    x = np.concatenate([logits_for("flat", 32, n, 51), logits_for("tied", 32, n, 52)])
    words = inputs.splitmix_u32(24, 0, 64)
    check(u, x, "f32", words, dict(top_p=p))
    check(u, x, "f32", words, dict(min_p=p, top_p=p[::-1].copy()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [5003, 40001, 300007])
def test_ties_that_most_warps_do_not_hold(u, n, dtype):
    """Cuts among long ties that lie in the middle or at the end of the row,
    all else far below: the warps without one are done with the search for
    the tie at once, while the others still read its key."""
    rows = 24
    rng = np.random.default_rng(n)
    x = np.full((rows, n), -90.0, np.float32)
    for b in range(rows):
        first = (n // 2, n - 2400)[b % 2]
        x[b, first : first + 2400] = 7.25 + 0.5 * (b % 3)  # positive: their keys' last digits are zero
    words = inputs.splitmix_u32(25, 0, rows)
    k = rng.choice([2, 40, 1000, 2047, 2399], rows).astype(np.int32)
    dev, held = as_type(x, dtype)
    for params in (dict(top_k=k), dict(top_p=rng.choice([0.01, 0.5, 0.999], rows).astype(np.float32)),
                   dict(top_k=k, top_p=np.full(rows, 0.6, np.float32))):
        want = oracle.sample_tokens(held, words, **params)
        for _ in range(20):
            got = run(u, dev, words, params)
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [1, 2])
@pytest.mark.parametrize("n,near", [(5003, 1), (40001, 38001), (100003, 700), (3001, 1500)])
def test_weights_last_octave(u, n, near, scale, dtype):
    """Logits whose distance is 31 exactly weigh 1, those past it nothing:
    `near` logits weigh more, the rest 1 or nothing, and top-k ends before, at
    and after the last of the heavy ones. With a temperature of log2 e (or half
    of it) the scale is exactly 1 (or 2). Words at both ends of the range, where
    the lightest tokens are drawn."""
    t = np.float32(float.fromhex("0x1.715476p+0") / scale)
    words = np.array([0, 1, 2, 38, 39, 1 << 31, 2**32 - 40, 2**32 - 2, 2**32 - 1], dtype=np.uint32)
    last = np.float32(-31.0 / scale)
    below, above = np.nextafter(last, np.float32(-99)), np.nextafter(last, np.float32(0))
    x = np.full((4, n), last, np.float32)
    x[1, n // 2 :] = below
    x[2, ::2] = above
    x[3, ::3], x[3, 1::3] = above, below
    rng = np.random.default_rng(n)
    for b, kind in enumerate(("front", "back", "apart", "apart")):
        at = {"front": np.arange(near), "back": np.arange(n - near, n), "apart": rng.permutation(n)[:near]}[kind]
        x[b, at] = 0.0
    x = np.repeat(x, words.size, 0)
    words = np.tile(words, 4)
    rows = words.size
    ks = [40, near, near + 1, min(n - 1, 3000), n - 1]
    for k in ks:
        k = np.full(rows, k, np.int32)
        filters = dict(temperature=np.full(rows, t), top_k=k)
        check(u, x, dtype, words, filters)
        check(u, x, dtype, words, dict(filters, top_p=np.full(rows, 0.9999999, np.float32)))
        check(u, x, dtype, words, dict(filters, min_p=np.full(rows, 2.0**-31, np.float32)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("stride", [2**32, 2**33 + 1, 2**40])
def test_the_stride_of_one_row_is_not_used(u, stride, dtype):
    """A view of one row may have any stride (say, one row of a wide buffer)."""
    x = logits_for("peaked", 1, 5003, 5)
    dev, held = as_type(x, dtype)
    view = dev.as_strided((1, 5003), (stride, 1))
    words, params = inputs.splitmix_u32(26, 0, 1), params_for("top_p", 1, 5)
    got, want = run(u, view, words, params), oracle.sample_tokens(held, words, **params)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_outputs_on_another_stream_while_the_current_one_is_busy(u):
    """The current stream gives memory back that it still writes to; a call on
    another stream gets none of it."""
    n, rows = 5003, 128
    x = logits_for("peaked", rows, n, 71)
    dev, held = as_type(x, "bf16")
    words = inputs.splitmix_u32(27, 0, rows)
    r = torch.from_numpy(words.view(np.int32).copy()).cuda()
    want = oracle.sample_tokens(held, words)
    side, current = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(current):
            torch.cuda._sleep(20_000_000)  # some 10 ms
            scratch = [torch.full((rows,), 12345, dtype=torch.int32, device="cuda") for _ in range(8)]
            del scratch
            tok, prob = u.sample_tokens(dev, r, stream=side)
        torch.cuda.synchronize()
        assert np.array_equal(tok.cpu().numpy(), want[0]) and np.array_equal(prob.cpu().numpy(), want[1])
