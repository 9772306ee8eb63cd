"""GPU tests of the language-model operators against plain 64-bit forms."""
import ctypes

import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp
import lm_ref as R
import oracle as O

pytestmark = pytest.mark.gpu

FT = [torch.float32, torch.float16, torch.bfloat16]
IT = [torch.uint8, torch.int8, torch.int32, torch.int64]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def random_desc(rng, n_states, n_groups, invalid):
    d = pp.DfaDesc()
    d.n_states, d.n_groups, d.background_group = n_states, n_groups, 0xFF
    d.invalid_state = n_states - 1 if invalid else 0xFF
    d.accept_mask = int(rng.integers(1, 1 << n_states))
    for b in range(256):
        d.byte_to_group[b] = int(rng.integers(0, n_groups))
    for g in range(n_groups):
        for s in range(n_states):
            sticky = rng.random() < 0.3  # so that some states lead nowhere
            d.delta[g][s] = s if sticky else int(rng.integers(0, n_states))
            if invalid and s == n_states - 1:
                d.delta[g][s] = s
    return d


DESCS = {
    "csv": lambda: pp.desc_csv(),
    "csv;": lambda: pp.desc_csv(b";", b"\n", b"'"),
    "crlf": lambda: pp.desc_csv_crlf(),
    "json": lambda: pp.desc_json_lexer(),
    "one": lambda: random_desc(np.random.default_rng(1), 1, 1, False),
    "seven": lambda: random_desc(np.random.default_rng(2), 7, 5, True),
    "sixteen": lambda: random_desc(np.random.default_rng(3), 16, 16, False),
    "dead": lambda: random_desc(np.random.default_rng(5), 16, 3, True),
}


def random_tokens(rng, n, sizes=(0, 12)):
    pool = np.frombuffer(b'abc012 \n\t,;"\'{}[]:\\.-+eE\r\xc3\xa9', np.uint8)
    out = []
    for _ in range(n):
        k = int(rng.integers(sizes[0], sizes[1]))
        free = rng.random() < 0.3
        b = rng.integers(0, 256, k).astype(np.uint8) if free else pool[rng.integers(0, pool.size, k)]
        out.append(bytes(b))
    return out


def column(tokens, base=0):
    """Arrow offsets and chars, the first token beginning at `base`."""
    off = np.zeros(len(tokens) + 1, np.int32)
    off[1:] = np.cumsum([len(t) for t in tokens])
    chars = np.frombuffer(b"\x00" * base + b"".join(tokens), np.uint8).copy()
    return dev(off + base), dev(chars)


def unpack(g):
    v = g.vectors.cpu().numpy().view(np.uint64)
    to = np.stack([(v >> np.uint64(4 * s)) & np.uint64(15) for s in range(16)], 1).astype(int)
    bits = np.unpackbits(g.allowed.cpu().numpy().view(np.uint8), axis=1, bitorder="little")
    return to, bits.astype(bool)


# ------------------------------------------------------------------ vocabularies
def check_vocab(tokens, desc, end=None, base=0):
    g = pp.vocab_grammar(*column(tokens, base), desc, end_id=end)
    to, bits = unpack(g)
    rto, rfine = R.vocab(tokens, desc, end)
    assert np.array_equal(to[:, :desc.n_states], rto)
    assert np.array_equal(to[:, desc.n_states:], np.tile(np.arange(desc.n_states, 16), (len(tokens), 1)))
    assert np.array_equal(bits[:, :len(tokens)], rfine)
    assert not bits[:, len(tokens):].any()
    return g


@pytest.mark.parametrize("kind", DESCS)
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 255, 256, 257, 1000])
def test_vocab(kind, n):
    rng = np.random.default_rng(n)
    check_vocab(random_tokens(rng, n), DESCS[kind](), end=n - 1 if n % 2 else None, base=n % 3)


@pytest.mark.parametrize("kind", ["csv", "json", "dead"])
@pytest.mark.parametrize("size", [62, 63, 64, 65, 95, 96, 97, 1000, 5001])
def test_vocab_long_tokens(kind, size):
    rng = np.random.default_rng(size)
    tokens = random_tokens(rng, 70)
    for v in (0, 5, 31, 32, 33, 69):
        tokens[v] = random_tokens(rng, 1, (size, size + 1))[0]
    check_vocab(tokens, DESCS[kind]())


def test_vocab_agrees_with_the_oracle():
    rng = np.random.default_rng(4)
    tokens = random_tokens(rng, 300) + [b"plain", b"12.5e-3", b'"q, x"', b"\n"]
    for kind, desc in ((O.KIND_CSV, pp.desc_csv()), (O.KIND_LEX, pp.desc_json_lexer())):
        to, _ = unpack(pp.vocab_grammar(*column(tokens), desc))
        for v, t in enumerate(tokens):
            assert list(to[v, :desc.n_states]) == list(O.stv(t, kind=kind)), (kind, t)


def test_vocab_end_token_with_bytes():
    tokens = [b"a", b'"', b"<end>", b""]
    g = check_vocab(tokens, pp.desc_csv(), end=2)
    assert g.accepts(torch.arange(8, device="cuda")).tolist() == [True, True, False, True] + [False] * 4


def test_vocab_bad_ranges_count_as_empty():
    off = dev(np.array([0, 3, -1, 4, 2, 9, 5, 6], np.int32))  # only 0 and 6 are ranges inside the chars
    chars = dev(np.frombuffer(b"abcdef", np.uint8).copy())
    to, bits = unpack(pp.vocab_grammar(off, chars, pp.desc_csv()))
    assert list(bits[0, :7]) == [True, False, False, False, False, False, True]
    for v in (1, 2, 3, 4, 5):
        assert list(to[v]) == list(range(16))


def test_vocab_writes_no_further_than_stated():
    """A stride beyond the next 256 tokens keeps what is there."""
    tokens = [b"x"] * 300
    off, chars = column(tokens)
    d = pp.desc_csv()
    vec = torch.empty(300, dtype=torch.int64, device="cuda")
    for stride in (10, 11, 16, 40):
        allowed = torch.full((5, stride), -7, dtype=torch.int32, device="cuda")
        rc = pp.lib().pp_vocab_grammar(off.data_ptr(), chars.data_ptr(), 300, 300, ctypes.byref(d), -1,
                                       vec.data_ptr(), allowed.data_ptr(), stride,
                                       torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        a = allowed.cpu().numpy()
        assert (a[:, 16:] == -7).all() and (a[:, 10:16] == 0).all()


def test_vocab_of_a_parsed_column():
    """The vocabulary as a string column that pp_parse wrote."""
    text = b'id,1\n"say ""x""",2\n"a,b",3\n'
    d_in = dev(np.frombuffer(text, np.uint8).copy())
    ((off, chars), ids), st = pp.parse_csv(d_in, ["str", "i32"])
    assert st["error"] == 0
    to, bits = unpack(pp.vocab_grammar(off, chars, pp.desc_csv()))
    rto, rfine = R.vocab([b"id", b'say "x"', b"a,b"], pp.desc_csv())
    assert np.array_equal(to[:, :5], rto) and np.array_equal(bits[:, :3], rfine)


def test_vocab_empty():
    g = pp.vocab_grammar(dev(np.zeros(1, np.int32)), dev(np.zeros(0, np.uint8)))
    assert g.vectors.numel() == 0 and g.allowed.shape == (5, 0)


# ------------------------------------------------------------------ states
def make_grammar(kind, n=200, seed=0):
    rng = np.random.default_rng(seed)
    tokens = random_tokens(rng, n, (0, 4))
    desc = DESCS[kind]()
    g = pp.vocab_grammar(*column(tokens), desc)
    return g, R.vocab(tokens, desc)[0], desc


@pytest.mark.parametrize("kind", ["csv", "json", "one", "sixteen"])
@pytest.mark.parametrize("cols", [0, 1, 2, 7, 15, 16, 17, 31, 33, 255, 257, 2047, 2048, 2049, 5000])
def test_states(kind, cols):
    g, to, desc = make_grammar(kind)
    rng = np.random.default_rng(cols)
    rows = 9
    # tokens that keep their states alive, and in some rows any
    calm = np.nonzero((to != (desc.invalid_state if desc.invalid_state != 255 else -1)).all(1))[0]
    calm = calm if calm.size else np.arange(200)
    tokens = calm[rng.integers(0, calm.size, (rows, cols))]
    tokens[::3] = rng.integers(0, 200, tokens[::3].shape)
    if cols > 3:
        tokens[4, cols // 2] = 200  # outside the vocabulary
        tokens[5, cols - 1] = -1
        tokens[6, 0] = 1 << 20
    start = rng.integers(0, desc.n_states, rows).astype(np.uint8)
    start[7] = 255
    start[8] = desc.n_states
    lengths = rng.integers(0, cols + 1, rows).astype(np.int32)
    lengths[:3] = [-5, cols + 10, cols]
    full = np.full(rows, cols)
    t = dev(tokens.astype(np.int32))
    got = pp.grammar_states(g, t, start=dev(start), lengths=dev(lengths)).cpu().numpy()
    assert np.array_equal(got, R.states(to, tokens, desc.n_states, start, lengths))
    got = pp.grammar_states(g, t).cpu().numpy()
    assert np.array_equal(got, R.states(to, tokens, desc.n_states, np.full(rows, desc.start_state), full))


@pytest.mark.parametrize("dtype", IT)
@pytest.mark.parametrize("cols", [3, 40, 2100])
def test_states_types_strides_and_continuation(dtype, cols):
    g, to, desc = make_grammar("json", n=120)
    rng = np.random.default_rng(7)
    tokens = rng.integers(0, 120, (5, cols))
    wide = dev(np.concatenate([tokens, tokens], 1)).to(dtype)
    t = wide[:, :cols]  # rows further apart than they are long
    start = np.array([0, 3, 4, 9, 2], np.uint8)
    ref = R.states(to, tokens, desc.n_states, start, np.full(5, cols))
    pad = torch.full((5, cols + 6), 77, dtype=torch.uint8, device="cuda")
    got = pp.grammar_states(g, t, start=dev(start), out=pad[:, 2:cols + 3])
    assert np.array_equal(got.cpu().numpy(), ref)
    assert (pad[:, :2] == 77).all() and (pad[:, cols + 3:] == 77).all()
    # the same in two calls: the second starts from the first one's last column
    one = pp.grammar_states(g, t[:, :cols // 2], start=dev(start))
    two = pp.grammar_states(g, t[:, cols // 2:], start=one[:, -1])
    assert np.array_equal(torch.cat([one[:, :-1], two], 1).cpu().numpy(), ref)


@pytest.mark.parametrize("rows,cols", [(1, 70001), (3, 40000), (700, 1), (300, 16), (200, 17), (1, 400000),
                                       (339, 17), (340, 17), (2001, 90), (5000, 250)])
def test_states_many(rows, cols):
    g, to, desc = make_grammar("csv", n=3000, seed=2)
    rng = np.random.default_rng(3)
    calm = np.nonzero((to[:, :4] != 4).all(1))[0]
    calm = calm if calm.size else np.nonzero((to[:, [0, 1, 2]] != 4).all(1))[0]
    quote = np.nonzero((to[:, 2] == 3) & (to[:, 3] == 2))[0]  # tokens of one quote
    tokens = calm[rng.integers(0, calm.size, (rows, cols))]
    if quote.size:
        at = rng.random((rows, cols)) < 0.01
        tokens[at] = quote[0]
    start = rng.integers(0, 4, rows).astype(np.uint8)
    # a vectorised walk over the columns
    ref = np.zeros((rows, cols + 1), np.uint8)
    ref[:, 0] = now = start
    for t in range(cols):
        now = to[tokens[:, t], now]
        ref[:, t + 1] = now
    got = pp.grammar_states(g, dev(tokens.astype(np.int32)), start=dev(start)).cpu().numpy()
    assert np.array_equal(got, ref)


# ------------------------------------------------------------------ logits
def logit_case(rng, rows, vocab, dtype, hist=20, n_bias=6):
    x = torch.from_numpy(rng.normal(0, 3, (rows, vocab))).to(dtype)
    c = {}
    if hist is not None:
        c["history"] = rng.integers(0, vocab, (rows, hist)).astype(np.int32)
        if hist:
            c["history"][:, ::2] = rng.integers(0, min(vocab, 5), c["history"][:, ::2].shape)
        c["history_len"] = rng.integers(0, hist + 1, rows).astype(np.int32)
        c["prompt_len"] = rng.integers(0, hist + 1, rows).astype(np.int32)
        c["repetition"] = rng.uniform(0.7, 1.6, rows).astype(np.float32)
        c["presence"] = rng.uniform(-1, 1, rows).astype(np.float32)
        c["frequency"] = rng.uniform(-0.5, 0.5, rows).astype(np.float32)
    if n_bias is not None:
        count = rng.integers(0, n_bias + 1, rows)
        at = np.zeros(rows + 1, np.int32)
        at[1:] = np.cumsum(count)
        tokens = rng.integers(0, vocab, at[-1]).astype(np.int32)  # some twice
        c["bias"] = (at, tokens, rng.normal(0, 5, at[-1]).astype(np.float32))
    return x, c


def on_gpu(c):
    return {k: tuple(dev(a) for a in v) if isinstance(v, tuple) else dev(v) for k, v in c.items()}


def random_grammar(rng, vocab, n_states=5):
    """A Grammar of random masks (the vectors play no part here)."""
    fine = rng.random((n_states, vocab)) < np.array([0.5, 0.02, 1.1, 0.0, 0.9])[:n_states, None]
    words = -(-vocab // 128) * 4
    bits = np.zeros((n_states, words * 32), np.uint8)
    bits[:, :vocab] = fine
    allowed = dev(np.packbits(bits, axis=1, bitorder="little").view(np.int32))
    g = pp.Grammar(torch.zeros(vocab, dtype=torch.int64, device="cuda"), allowed, vocab, pp.desc_csv())
    return g, fine


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 33, 127, 1000, 1025, 2049, 4096, 4097, 33001])
def test_logits_everything(dtype, vocab):
    rng = np.random.default_rng(vocab)
    rows = 11
    x, c = logit_case(rng, rows, vocab, dtype, hist=50, n_bias=9)
    g, fine = random_grammar(rng, vocab)
    states = rng.integers(0, 5, rows).astype(np.uint8)
    states[:5] = [0, 1, 2, 3, 4]
    states[9:] = [5, 255]  # states that the grammar does not have
    mask = np.stack([fine[s] if s < 5 else np.zeros(vocab, bool) for s in states])
    got = pp.process_logits(x.cuda(), grammar=g, states=dev(states), **on_gpu(c))
    ref, error = R.logits(x.double().numpy(), fine=mask, **c)
    R.check(got, ref, error, dtype)
    assert torch.isinf(got[3]).all() and torch.isinf(got[9]).all()  # rows without any token


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("what", ["history", "bias", "mask", "history bias", "history mask", "bias mask", ""])
def test_logits_parts(dtype, what):
    rng = np.random.default_rng(len(what))
    rows, vocab = 6, 5003
    x, c = logit_case(rng, rows, vocab, dtype, 30 if "history" in what else None, 8 if "bias" in what else None)
    kw, mask = {}, None
    if "mask" in what:
        g, fine = random_grammar(rng, vocab)
        states = rng.integers(0, 5, rows).astype(np.uint8)
        kw, mask = dict(grammar=g, states=dev(states)), fine[states]
    ref, error = R.logits(x.double().numpy(), fine=mask, **c)
    R.check(pp.process_logits(x.cuda(), **on_gpu(c), **kw), ref, error, dtype)


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("shift,gap,oshift,ogap,place", [
    (0, 0, 0, 0, "other"), (1, 0, 1, 0, "other"), (3, 5, 3, 5, "same"), (0, 3, 0, 3, "same"),
    (1, 2, 0, 2, "other"), (2, 1, 2, 0, "other"), (7, 8, 7, 16, "other")])
def test_logits_strides_and_alignment(dtype, shift, gap, oshift, ogap, place):
    rng = np.random.default_rng(shift * 10 + gap)
    rows, vocab = 5, 2051
    x, c = logit_case(rng, rows, vocab, dtype)
    g, fine = random_grammar(rng, vocab)
    states = rng.integers(0, 5, rows).astype(np.uint8)

    def strided(shift, gap, fill):
        buf = torch.full((shift + rows * (vocab + gap) + 16,), fill, dtype=dtype, device="cuda")
        return buf, buf[shift:shift + rows * (vocab + gap)].view(rows, vocab + gap)[:, :vocab]

    buf, src = strided(shift, gap, 5.0)
    src.copy_(x)
    obuf, out = (buf, src) if place == "same" else strided(oshift, ogap, 7.0)
    got = pp.process_logits(src, grammar=g, states=dev(states), out=out, **on_gpu(c))
    assert got.data_ptr() == out.data_ptr()
    ref, error = R.logits(x.double().numpy(), fine=fine[states], **c)
    R.check(got, ref, error, dtype)
    fill = 5.0 if place == "same" else 7.0
    out.fill_(fill)  # nothing around the rows was written
    assert (obuf == fill).all()


def test_logits_history_rows_lengths_and_tokens_outside():
    """Several rows of one sequence (a draft's positions), lengths below zero
    and past the history, history rows and tokens that do not exist."""
    rng = np.random.default_rng(8)
    rows, vocab = 9, 700
    for dtype in IT:
        x, _ = logit_case(rng, rows, vocab, torch.float32, None, None)
        top = {torch.uint8: 256, torch.int8: 128}.get(dtype, 900)
        history = rng.integers(0 if dtype == torch.uint8 else -20, top, (2, 64))
        c = {"history": history, "history_row": np.array([0, 0, 0, 1, 1, 1, 2, -1, 1], np.int32),
             "history_len": np.array([3, 4, 5, -2, 64, 99, 64, 64, 0], np.int32),
             "prompt_len": np.array([3, 3, 3, 0, -9, 70, 0, 0, 0], np.int32),
             "repetition": rng.uniform(0.5, 2, rows).astype(np.float32),
             "presence": np.ones(rows, np.float32), "frequency": np.full(rows, 0.25, np.float32)}
        ref, error = R.logits(x.double().numpy(), **c)
        kw = on_gpu(c)
        wide = torch.zeros(2, 80, dtype=dtype, device="cuda")
        wide[:, :64] = kw["history"].to(dtype)
        kw["history"] = wide[:, :64]
        R.check(pp.process_logits(x.cuda(), **kw), ref, error, torch.float32)


def test_logits_bias_entries_outside_and_repeated():
    x = np.zeros((3, 40))
    at = np.array([-3, 4, 4, 99], np.int32)
    tokens = np.array([7, -1, 40, 7, 5, 6, 5], np.int32)
    values = np.array([1, 2, 3, 4, 5, 6, 7], np.float32)
    got = pp.process_logits(dev(x, torch.float32), bias=(dev(at), dev(tokens), dev(values))).cpu().numpy()
    want = np.zeros((3, 40))
    want[0, 7], want[2, 5], want[2, 6] = 4, 7, 6  # the last entry of a token counts
    assert np.array_equal(got, want)


@pytest.mark.parametrize("hist", [20, 40000])
def test_logits_long_bias_lists(hist):
    """Lists of more entries than 16 bits count, with every token twice; with
    a short history and one that needs counts of more than 15 bits."""
    rng = np.random.default_rng(11)
    vocab = 50000
    tokens = np.concatenate([rng.permutation(vocab), rng.permutation(vocab)[:49000], [7, 7]]).astype(np.int32)
    values = rng.normal(0, 3, tokens.size).astype(np.float32)
    x = rng.normal(0, 2, (3, vocab)).astype(np.float32)
    c = {"bias": (np.array([0, 5, 5, tokens.size], np.int32), tokens, values),
         "history": rng.integers(0, 300, (3, hist)).astype(np.int32),
         "frequency": np.full(3, 0.125, np.float32)}
    ref, error = R.logits(x, **c)
    R.check(pp.process_logits(dev(x), **on_gpu(c)), ref, error, torch.float32)


@pytest.mark.parametrize("dtype", FT)
def test_logits_infinities_and_nan(dtype):
    rng = np.random.default_rng(9)
    vocab = 2500
    x, c = logit_case(rng, 5, vocab, dtype, hist=40)
    low = torch.finfo(dtype).min
    x[:, 0::50] = float("nan")
    x[:, 1::50] = float("inf")
    x[:, 2::50] = -float("inf")
    x[:, 3::50] = low
    c["history"][:, :8] = [0, 1, 2, 3, 50, 51, 52, 53]
    c["history_len"][:] = 40
    c["repetition"][:] = 1.0  # the lowest value stays in range
    c["presence"][:] = 0.5
    c["frequency"][:] = 0.0
    g, fine = random_grammar(rng, vocab)
    states = np.array([0, 1, 2, 3, 4], np.uint8)
    got = pp.process_logits(x.cuda(), grammar=g, states=dev(states), **on_gpu(c))
    with np.errstate(invalid="ignore"):
        ref, error = R.logits(x.double().numpy(), fine=fine[states], **c)
    error[~np.isfinite(error)] = 0
    R.check(got, ref, error, dtype)


def test_logits_rounding_past_the_range():
    """What leaves the type's range becomes infinite, as any rounding does."""
    x = torch.tensor([[60000.0, -60000.0, 1.0]], dtype=torch.float16, device="cuda")
    got = pp.process_logits(x, bias=(dev(np.array([0, 2], np.int32)), dev(np.array([0, 1], np.int32)),
                                     dev(np.array([9000, -9000], np.float32))))
    assert got.tolist() == [[float("inf"), -float("inf"), 1.0]]


def test_logits_long_history_counts_exactly():
    """More repetitions than 16 bits hold, from every thread at once."""
    n, vocab = 200000, 3000
    history = np.zeros((2, n), np.int32)
    history[1] = np.arange(n) % vocab
    x = np.zeros((2, vocab))
    one = np.ones(2, np.float32)
    got = pp.process_logits(dev(x, torch.float32), history=dev(history), frequency=dev(one),
                            prompt_len=dev(np.array([1000, 0], np.int32))).cpu().numpy()
    assert got[0, 0] == -(n - 1000) and (got[0, 1:] == 0).all()
    assert np.array_equal(got[1], -np.bincount(history[1], minlength=vocab).astype(float))


@pytest.mark.parametrize("n", [65535, 65536])
def test_logits_counts_at_16_bits(n):
    """One token alone, beside one that is never said, at both widths of the
    counts."""
    history = np.full((2, n), 5, np.int32)
    history[1] = 4
    got = pp.process_logits(dev(np.zeros((2, 1100)), torch.float32), history=dev(history),
                            frequency=dev(np.ones(2, np.float32))).cpu().numpy()
    want = np.zeros((2, 1100))
    want[0, 5], want[1, 4] = -n, -n
    assert np.array_equal(got, want)


@pytest.mark.parametrize("rows,vocab", [(1, 200000), (70000, 9), (3000, 257)])
def test_logits_shapes(rows, vocab):
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.normal(0, 3, (rows, vocab))).to(torch.bfloat16)
    history = rng.integers(0, vocab, (rows, 12)).astype(np.int32)
    rep = rng.uniform(1, 2, rows).astype(np.float32)
    g, fine = random_grammar(rng, vocab)
    states = rng.integers(0, 5, rows).astype(np.uint8)
    got = pp.process_logits(x.cuda(), history=dev(history), repetition=dev(rep), grammar=g, states=dev(states))
    y = x.double().numpy()
    seen = np.zeros((rows, vocab), bool)
    np.put_along_axis(seen, history.astype(np.int64), True, 1)
    r = rep[:, None].astype(np.float64)
    y = np.where(seen, np.where(y > 0, y / r, y * r), y)
    y[~fine[states]] = -np.inf
    R.check(got, y, np.where(np.isfinite(y), 2 * R.U32 * np.abs(y), 0), torch.bfloat16)


def test_logits_offsets_past_32_bits():
    rows, vocab = 17000, 131075  # 2.2 billion logits
    x = torch.full((rows, vocab), 2.0, dtype=torch.bfloat16, device="cuda")
    history = torch.arange(rows, device="cuda", dtype=torch.int32)[:, None]
    got = pp.process_logits(x, history=history, repetition=torch.full((rows,), 2.0, device="cuda"), out=x)
    for r in (0, 1, 16383, 16384, 16999):
        line = got[r].cpu()
        assert line[r] == 1.0 and (line == 2.0).sum() == vocab - 1


# ------------------------------------------------------------------ embedding
def ids_of(rng, n, vocab, dtype):
    top = {torch.uint8: 256, torch.int8: 128}.get(dtype, 1 << 30)
    ids = rng.integers(0, min(vocab, top), n)
    if n > 4:
        ids[1] = min(vocab, top - 1)  # outside the table, where the type reaches
        ids[2] = 3 % vocab
        if dtype != torch.uint8:
            ids[3] = -1
    return ids


@pytest.mark.parametrize("out", FT)
@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 9, 64, 257, 1000, 2056])
def test_embed(dtype, out, dim):
    rng = np.random.default_rng(dim)
    n, vocab = 301, 77
    table = torch.from_numpy(rng.normal(0, 1, (vocab, dim))).to(dtype)
    ids = ids_of(rng, n, vocab, torch.int32)
    got = pp.embed(dev(ids.astype(np.int32)), table.cuda(), scale=1.7, padding_id=3, dtype=out)
    ref = R.embed(ids, table.double().numpy(), 1.7, 3)
    R.check(got, ref, R.U32 * np.abs(ref), out)


@pytest.mark.parametrize("dtype", IT)
def test_embed_ids(dtype):
    """Id types, shapes, strides (also 0) and an empty list; table rows apart."""
    rng = np.random.default_rng(2)
    vocab, dim = 90, 24
    wide = torch.from_numpy(rng.normal(0, 1, (vocab, 32))).float().cuda()
    for table in (wide[:, :dim], wide[:, 3:3 + dim], wide[:, :dim].to(torch.bfloat16)):
        t = table.double().cpu().numpy()
        ids = ids_of(rng, 60, vocab, dtype)
        d = dev(ids).to(dtype)
        ids = d.cpu().numpy().astype(np.int64)
        got = pp.embed(d.view(3, 4, 5), table)
        assert got.shape == (3, 4, 5, dim)
        assert np.array_equal(got.double().cpu().numpy().reshape(60, dim), R.embed(ids, t, 1, None))
        got = pp.embed(d[::3], table)
        assert np.array_equal(got.double().cpu().numpy(), R.embed(ids[::3], t, 1, None))
        got = pp.embed(d[7:8].expand(9), table, padding_id=None)
        assert np.array_equal(got.double().cpu().numpy(), R.embed(ids[7:8].repeat(9), t, 1, None))
        assert pp.embed(d[:0], table).shape == (0, dim)
    out = torch.full((62, dim), 9.0, device="cuda")
    pp.embed(d, wide[:, :dim], out=out[1:61])
    assert (out[0] == 9).all() and (out[61] == 9).all()


def test_embed_offsets_past_32_bits():
    vocab, dim = 600000, 4096
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    table[-1], table[1] = 3.0, 1.0
    ids = torch.tensor([vocab - 1, 1, 0], device="cuda")
    assert pp.embed(ids, table)[:, ::511].float().unique(dim=1).flatten().tolist() == [3.0, 1.0, 0.0]
    grad = torch.ones(3, dim, dtype=torch.bfloat16, device="cuda")
    pp.embed_grad(ids, grad, vocab, out=table)
    assert table[-1].float().min() == 1.0 and table[1].float().max() == 1.0
    assert table[2:-1].abs().max() == 0


GRAD_N = [0, 1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 257, 383, 384, 385, 512, 1000, 4095, 4096, 4097, 9000]


def grad_ids(rng, n, vocab, how):
    if how == "any":
        ids = rng.integers(0, vocab, n)
    elif how == "one":
        ids = np.full(n, min(vocab - 1, 5))
    elif how == "few":
        ids = rng.integers(0, min(vocab, 3), n)
    elif how == "zipf":
        ids = np.minimum(rng.zipf(1.3, n) - 1, vocab - 1)
    elif how == "outside":
        ids = np.where(rng.random(n) < 0.5, -1, vocab)
    else:  # runs whose lengths straddle the chunks' ends
        ids = np.repeat(np.arange(vocab), 61)[:n]
        ids = rng.permutation(np.resize(ids, n))
    return ids


@pytest.mark.parametrize("how", ["any", "one", "few", "zipf", "outside", "runs"])
@pytest.mark.parametrize("n", GRAD_N)
def test_grad_ids(n, how):
    rng = np.random.default_rng(n)
    vocab, dim = 300, 40
    ids = grad_ids(rng, n, vocab, how)
    grad = torch.from_numpy(rng.normal(0, 1, (n, dim))).float()
    got = pp.embed_grad(dev(ids.astype(np.int32)), grad.cuda(), vocab, scale=0.5, padding_id=2)
    ref, error = R.embed_grad(ids, grad.double().numpy(), vocab, 0.5, 2)
    R.check(got, ref, error, torch.float32)
    again = pp.embed_grad(dev(ids.astype(np.int32)), grad.cuda(), vocab, scale=0.5, padding_id=2)
    assert torch.equal(got, again)


@pytest.mark.parametrize("how", ["zipf", "runs", "one"])
@pytest.mark.parametrize("n", [1024, 1025, 8192, 8193, 16384, 16385, 32769, 65537, 131072, 131073, 140001, 262144, 400003])
def test_grad_many_ids(n, how):
    """The sizes at which another sort takes over, and their neighbours."""
    rng = np.random.default_rng(n)
    vocab, dim = 2500, 12
    ids = grad_ids(rng, n, vocab, how)
    ids[::1000] = -1
    grad = rng.normal(0, 1, (n, dim)).astype(np.float32)
    for accumulate in (False, True):
        old = rng.normal(0, 1, (vocab, dim)).astype(np.float32)
        got = pp.embed_grad(dev(ids), dev(grad), vocab, out=dev(old), accumulate=accumulate)
        ref, size, count = np.zeros((vocab, dim)), np.zeros((vocab, dim)), np.zeros(vocab)
        ok = ids >= 0
        np.add.at(ref, ids[ok], grad[ok].astype(np.float64))
        np.add.at(size, ids[ok], np.abs(grad[ok]).astype(np.float64))
        np.add.at(count, ids[ok], 1)
        error = (count[:, None] + 2) * R.U32 * size
        if accumulate:
            ref = ref + old
            error = error + 2 * R.U32 * (np.abs(ref) + np.abs(old)) * (count[:, None] > 0)
        R.check(got, ref, error, torch.float32)


@pytest.mark.parametrize("dim", [256, 600, 601])
@pytest.mark.parametrize("first", [0, 1, 7])
@pytest.mark.parametrize("runs", [[500, 511, 512, 513, 520, 521, 529], [2016, 2047, 2048, 2049, 2080, 2081, 2113],
                                  [3, 16640, 1, 40000, 5, 16639], [120000], [20, 300000]])
def test_grad_of_long_runs(runs, first, dim):
    """Ids that so many positions name that blocks share their sums, and those just below."""
    rng = np.random.default_rng(first)
    ids = np.concatenate([np.full(first, 0)] + [np.full(k, 2 * i + 1) for i, k in enumerate(runs)])
    rng.shuffle(ids)
    grad = rng.integers(-8, 9, (len(ids), dim)).astype(np.float32)  # sums without rounding
    ref = np.zeros((2 * len(runs) + 3, dim))
    for i in np.unique(ids):
        ref[i] = grad[ids == i].sum(0, dtype=np.float64)
    got = pp.embed_grad(dev(ids), dev(grad).to(torch.bfloat16), len(ref), dtype=torch.float32)
    assert np.array_equal(got.cpu().numpy().astype(np.float64), ref)


@pytest.mark.parametrize("vocab", [1, 2, 255, 256, 257, 65535, 65536, 70000, 300000])
def test_grad_vocabularies(vocab):
    rng = np.random.default_rng(vocab)
    n, dim = 3000, 5
    ids = grad_ids(rng, n, vocab, "any")
    ids[:200] = vocab - 1
    grad = torch.from_numpy(rng.normal(0, 1, (n, dim))).float()
    got = pp.embed_grad(dev(ids), grad.cuda(), vocab)
    ref, error = R.embed_grad(ids, grad.double().numpy(), vocab, 1, -1)
    R.check(got, ref, error, torch.float32)


@pytest.mark.parametrize("n", [100, 700])
@pytest.mark.parametrize("out", FT)
@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("dim", [1, 7, 8, 9, 63, 64, 65, 255, 256, 257, 1000, 2051])
def test_grad_types_and_widths(dtype, out, dim, n):
    rng = np.random.default_rng(dim)
    vocab = 90
    ids = grad_ids(rng, n, vocab, "zipf")
    ids[::7] = 11
    grad = torch.from_numpy(rng.normal(0, 1, (n, dim))).to(dtype)
    for accumulate in (False, True):
        old = torch.from_numpy(rng.normal(0, 1, (vocab, dim))).to(out)
        got = pp.embed_grad(dev(ids), grad.cuda(), vocab, scale=1.25, padding_id=0, out=old.cuda(), accumulate=accumulate)
        ref, error = R.embed_grad(ids, grad.double().numpy(), vocab, 1.25, 0, old.double().numpy() if accumulate else None)
        R.check(got, ref, error, out)
        if accumulate:  # rows of ids that do not occur are as they were
            gone = np.setdiff1d(np.arange(vocab), ids[ids != 0])
            assert torch.equal(got.cpu()[gone], old[gone])


@pytest.mark.parametrize("dtype", IT)
def test_grad_strides_and_shared_rows(dtype):
    rng = np.random.default_rng(5)
    n, vocab, dim = 200, 100, 24
    ids = ids_of(rng, 2 * n, vocab, dtype)
    d = dev(ids).to(dtype)[::2]
    host = d.cpu().numpy().astype(np.int64)
    wide = torch.from_numpy(rng.normal(0, 1, (n, 40))).float().cuda()
    whole = torch.full((vocab, 33), 4.0, device="cuda")
    for grad in (wide[:, :dim], wide[:, 5:5 + dim], wide[3:4, :dim].expand(n, dim)):
        got = pp.embed_grad(d, grad, vocab, out=whole[:, 4:4 + dim])
        ref, error = R.embed_grad(host, grad.double().cpu().numpy(), vocab, 1, -1)
        R.check(got, ref, error, torch.float32)
    assert (whole[:, :4] == 4).all() and (whole[:, 4 + dim:] == 4).all()


@pytest.mark.parametrize("n", [1, 300, 5000, 140000])
def test_grad_of_a_very_large_vocabulary(n):
    """More rows than a block looks at together, ids of 28 bits."""
    rng = np.random.default_rng(n)
    vocab = (1 << 27) + 3
    ids = rng.integers(0, vocab, n)
    ids[:min(n, 100)] = vocab - 1
    out = torch.full((vocab, 1), 9.0, device="cuda")
    pp.embed_grad(dev(ids), torch.ones(n, 1, device="cuda"), vocab, out=out, padding_id=int(ids[-1]) if n > 1 else None)
    keep = ids[ids != ids[-1]] if n > 1 else ids
    which, count = np.unique(keep, return_counts=True)
    at = torch.nonzero(out[:, 0]).flatten()
    assert np.array_equal(at.cpu().numpy(), which)
    assert np.array_equal(out[at, 0].cpu().numpy(), count.astype(np.float32))


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("dim", [1, 3, 5, 13, 37, 61, 127, 250])
def test_aligned_rows_of_odd_widths(dtype, dim):
    """Rows that begin on 16-byte boundaries and end anywhere: a table, a
    gradient and a result inside wider arrays."""
    rng = np.random.default_rng(dim)
    vocab = 60
    wide = torch.from_numpy(rng.normal(0, 1, (900, 256))).to(dtype).cuda()
    for n in (1, 50, 900):
        ids = grad_ids(rng, n, vocab, "zipf")
        table = wide[:vocab, :dim]
        got = pp.embed(dev(ids), table, scale=0.75)
        ref = R.embed(ids, table.double().cpu().numpy(), 0.75, None)
        R.check(got, ref, R.U32 * np.abs(ref), dtype)
        for out in (torch.float32, dtype):
            whole = torch.full((vocab, 256), 5.0, dtype=out, device="cuda")
            got = pp.embed_grad(dev(ids), wide[:n, :dim], vocab, out=whole[:, :dim])
            ref, error = R.embed_grad(ids, wide[:n, :dim].double().cpu().numpy(), vocab, 1, -1)
            R.check(got, ref, error, out)
            assert (whole[:, dim:] == 5).all()


def test_grad_through_autograd():
    rng = np.random.default_rng(6)
    vocab, dim, n = 17, 12, 50
    table = torch.from_numpy(rng.normal(0, 1, (vocab, dim))).float().cuda().requires_grad_()
    ids = dev(grad_ids(rng, n, vocab, "any").reshape(5, 10))
    weight = torch.from_numpy(rng.normal(0, 1, (5, 10, dim))).float().cuda()
    loss = (pp.embed(ids, table, scale=2.0, padding_id=4) * weight).sum()
    loss.backward()
    ref, error = R.embed_grad(ids.cpu().numpy().ravel(), weight.double().cpu().numpy().reshape(n, dim), vocab, 2.0, 4)
    R.check(table.grad, ref, error, torch.float32)
    # against differences: the sum is linear in the table, so a step of any
    # size gives the slope; each of the sums over n * dim products rounds
    base = table.detach()
    for v, c in ((int(ids[0, 0]), 3), (4, 0), (16, 11)):
        step = base.clone()
        step[v, c] += 0.5
        with torch.no_grad():
            up = (pp.embed(ids, step, scale=2.0, padding_id=4).double() * weight.double()).sum()
            down = (pp.embed(ids, base, scale=2.0, padding_id=4).double() * weight.double()).sum()
        slope = float((up - down) / 0.5)
        size = float((pp.embed(ids, step, scale=2.0, padding_id=4).double() * weight.double()).abs().sum())
        assert abs(slope - float(table.grad[v, c])) <= 8 * R.U32 * size + error[v, c]
    # a gradient that is one number for all
    table.grad = None
    pp.embed(ids, table).sum().backward()
    ref, error = R.embed_grad(ids.cpu().numpy().ravel(), np.ones((n, dim)), vocab, 1, -1)
    R.check(table.grad, ref, error, torch.float32)


def test_on_another_stream():
    """Every operator on a stream that is not the current one, from inputs
    made on it, several in flight."""
    s = torch.cuda.Stream()
    rng = np.random.default_rng(7)
    tokens = random_tokens(rng, 500)
    off, chars = column(tokens)
    ids = dev(rng.integers(0, 500, 4000).astype(np.int32))
    table = torch.randn(500, 64, device="cuda")
    x = torch.randn(4, 500, device="cuda")
    torch.cuda.synchronize()
    want = []
    for stream in (None, s, s):
        g = pp.vocab_grammar(off, chars, pp.desc_csv(), stream=stream)
        st = pp.grammar_states(g, ids.view(4, 1000), stream=stream)
        ctx = torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream())
        with ctx:
            now = st[:, 7]
        y = pp.process_logits(x, grammar=g, states=now, stream=stream)
        e = pp.embed(ids, table, stream=stream)
        d = pp.embed_grad(ids, e, 500, stream=stream)
        want.append((g.vectors, g.allowed, st, y, e, d))
    torch.cuda.synchronize()
    for other in want[1:]:
        for a, b in zip(want[0], other):
            assert torch.equal(a, b)


def test_in_a_graph():
    """A decode step's calls captured and replayed with other inputs."""
    rng = np.random.default_rng(8)
    tokens = random_tokens(rng, 600, (1, 4))
    g = pp.vocab_grammar(*column(tokens), pp.desc_csv())
    table = torch.randn(600, 32, device="cuda")
    x = torch.randn(3, 600, device="cuda")
    pick = torch.zeros(3, 1, dtype=torch.int64, device="cuda")
    first = torch.zeros(3, dtype=torch.uint8, device="cuda")

    def step():
        st = pp.grammar_states(g, pick, start=first)
        return st, pp.process_logits(x, history=pick, repetition=rep, grammar=g, states=st[:, 1]), \
            pp.embed(pick, table), pp.embed_grad(pick[:, 0], table[:3], 600)

    rep = torch.full((3,), 1.5, device="cuda")
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        pick.copy_(torch.from_numpy(rng.integers(0, 600, (3, 1))))
        x.normal_()
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_the_example_learns_and_answers_rows_that_parse():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "grammar_rows.py")
    spec = importlib.util.spec_from_file_location("grammar_rows", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    out = example.run()
    assert out["losses"][-1] < 0.6 * out["losses"][0] and out["same_states"]
    done = [p for p in out["parsed"] if p is not None]
    assert done and all(p["error"] & pp.ERR_FATAL == 0 for p in done)  # what the grammar lets end, parses
    assert all(p is not None for p, over in zip(out["parsed"], out["over"]) if over)
