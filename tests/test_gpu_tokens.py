"""GPU tests of the probabilities of tokens and of the verification of drafts
against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp
import tokens_ref as R

pytestmark = pytest.mark.gpu

FT = [torch.float32, torch.float16, torch.bfloat16]
IT = [torch.uint8, torch.int8, torch.int32, torch.int64]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def wide(t):
    return t.double().cpu().numpy()


def placed(rows, cols, dtype, stride, offset):
    """An empty [rows, cols] view at `offset` elements, rows `stride` apart, and what it lies in."""
    whole = torch.full((rows * stride + offset + 8,), 77, dtype=dtype, device="cuda")
    return torch.as_strided(whole, (rows, cols), (stride, 1), offset), whole


def check(got, x, t=None, k=None):
    ref, err = R.probs(wide(x), t, k)
    off = np.abs(wide(got) - ref)
    assert (off <= err).all(), (off - err).max()
    assert ((wide(got) == 0) | (ref > 0)).all()  # nothing but the kept tokens


def logits(rng, rows, vocab, dtype, gone=0.3):
    x = rng.normal(0, 3, (rows, vocab))
    x[rng.random((rows, vocab)) < gone] = -np.inf
    return dev(x, dtype)


# ------------------------------------------------------------ probabilities
@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 31), (5, 257), (4, 1000), (2, 4099), (3, 16384), (1, 32000),
                                        (2, 65537), (1, 131075), (700, 300), (40, 8192)])
def test_probs(dtype, rows, vocab):
    rng = np.random.default_rng(rows * 1000 + vocab)
    x = logits(rng, rows, vocab, dtype)
    t = rng.uniform(0.3, 2.0, rows).astype(np.float32)
    t[rng.random(rows) < 0.2] = 0
    k = np.minimum(np.exp(rng.uniform(0, np.log(vocab + 2), rows)), vocab + 1).astype(np.int32)
    check(pp.token_probs(x), x)
    check(pp.token_probs(x, temperature=dev(t)), x, t)
    check(pp.token_probs(x, top_k=dev(k)), x, None, k)
    check(pp.token_probs(x, temperature=dev(t), top_k=dev(k)), x, t, k)


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("offset,extra,out_offset", [(0, 0, 1), (1, 3, 0), (3, 1, 2), (5, 8, 3), (7, 5, 0)])
def test_probs_of_strided_and_unaligned_rows(dtype, offset, extra, out_offset):
    """Both ends of every row, and nothing written beside the result."""
    rng = np.random.default_rng(offset)
    for vocab in (1, 6, 129, 5000):
        x, _ = placed(5, vocab, dtype, vocab + extra, offset)
        x.copy_(logits(rng, 5, vocab, dtype))
        out, whole = placed(5, vocab, torch.float32, vocab + 3, out_offset)
        k = np.array([1, 2, 3, vocab, 0], np.int32)
        assert pp.token_probs(x, top_k=dev(k), out=out) is out
        check(out, x, None, k)
        there = torch.zeros_like(whole, dtype=torch.bool)
        torch.as_strided(there, (5, vocab), (vocab + 3, 1), out_offset).fill_(True)
        assert (whole[~there] == 77).all()


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("vocab", [7, 1000, 33000])
def test_probs_of_ties(dtype, vocab):
    """Few different values: of those that tie the lowest tokens stay, exactly k."""
    rng = np.random.default_rng(vocab)
    x = dev(rng.integers(-2, 3, (9, vocab)).astype(np.float64), dtype)
    x[8] = 1.5
    x[7] = torch.where(torch.arange(vocab, device="cuda") % 2 == 0, 0.0, -0.0)  # equal, whatever the sign
    k = np.array([1, 2, 3, vocab // 7, vocab // 3, vocab // 2, vocab - 1, vocab // 2, vocab - 2], np.int32)
    got = pp.token_probs(x, top_k=dev(k))
    check(got, x, None, k)
    assert ((got > 0).sum(1).cpu().numpy() == k).all()
    greedy = pp.token_probs(x, temperature=torch.zeros(9, device="cuda"))
    assert torch.equal(greedy.argmax(1), (x == x.max(1, keepdim=True).values).int().argmax(1)) and (greedy.sum(1) == 1).all()


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("vocab", [40, 9001])
def test_probs_of_masks_infinities_and_nan(dtype, vocab):
    inf, nan = np.inf, np.nan
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (10, vocab))
    x[0] = -inf
    x[1] = nan
    x[2, :] = -inf
    x[2, vocab - 1] = 3.0
    x[3, 5:9] = inf
    x[4, ::2] = nan
    x[5, ::3] = inf
    x[5, 1::3] = nan
    x[6] = torch.finfo(dtype).min
    x[7, 1:] = torch.finfo(dtype).min
    x[8] = torch.finfo(dtype).max
    x[9, ::2] = -inf
    x = dev(x, dtype)
    for t, k in ((None, None), (0.7, None), (0.0, None), (1.0, 3), (-1.0, 2), (nan, None), (1e-38, 4), (1e-44, None),
                 (inf, 2), (3e38, None), (1.0, -5), (1.0, 2 ** 31 - 1), (1.0, vocab), (1.0, vocab - 1)):
        tt = None if t is None else np.full(10, t, np.float32)
        kk = None if k is None else np.full(10, k, np.int32)
        got = wide(pp.token_probs(x, None if t is None else dev(tt), None if k is None else dev(kk)))
        assert np.isfinite(got).all()
        assert (got[0] == 0).all() and (got[1] == 0).all() and got[2, vocab - 1] == 1 and got[2].sum() == 1
        if t != inf:  # where no difference of infinities is divided by one
            check(dev(got), x, tt, kk)
        else:
            assert (got[9] > 0).sum() == 2 and np.allclose(got[9].max(), 0.5)


def test_probs_in_place_and_without_rows():
    x = logits(np.random.default_rng(2), 6, 5003, torch.float32)
    k = torch.tensor([3, 0, 40, 5002, 1, 600], dtype=torch.int32, device="cuda")
    want = pp.token_probs(x, top_k=k)
    assert pp.token_probs(x, top_k=k, out=x) is x and torch.equal(x, want)
    assert pp.token_probs(x[:0]).shape == (0, 5003) and pp.token_probs(x[:, :0]).shape == (6, 0)


@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 200001), (torch.float32, 420001), (torch.float16, 500000), (torch.bfloat16, 900001)])
def test_probs_of_rows_beyond_shared_memory(dtype, vocab):
    rng = np.random.default_rng(3)
    x = logits(rng, 2, vocab, dtype)
    for k in ([0, 0], [1000, 1], [vocab // 2, 5000]):
        k = np.array(k, np.int32)
        check(pp.token_probs(x, top_k=dev(k)), x, None, k)
    check(pp.token_probs(x, temperature=dev(np.array([0.5, 0.0], np.float32))), x, [0.5, 0.0])


def test_probs_past_32_bit_offsets():
    """The last rows of logits and of probabilities lie beyond 2^32 bytes, and 2^31 elements."""
    rows, vocab = 17000, 131072
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    last = logits(np.random.default_rng(4), 2, vocab, torch.bfloat16)
    x[-2:] = last
    k = torch.full((rows,), 100, dtype=torch.int32, device="cuda")
    got = pp.token_probs(x, top_k=k)
    check(got[-2:], last, None, [100, 100])
    assert (got[7] > 0).sum() == 100 and (got[7, :100] > 0).all()


def kinds_of_rows(rng, vocab):
    """Rows on which a cut takes each of its ways: values spread, alike, far from one another, few, masked."""
    x = rng.normal(0, 3, (9, vocab))
    x[1] = np.round(x[1])  # ties everywhere
    x[2] = 0.25
    x[3, vocab // 2] = -60000.0  # one far below, so that the others share a step
    x[4] = np.where(rng.random(vocab) < 0.97, -np.inf, x[4])
    x[5, ::2] = np.nan
    x[6] = np.arange(vocab) % 7 * 1e-3
    x[7, :3] = np.inf
    x[8] = np.exp(x[8])
    return x


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("vocab", [1500, 9000, 20011, 70001, 131075])
def test_probs_of_long_cuts(dtype, vocab):
    """Cuts of more than the lists of candidates hold, in clusters of one to eight blocks."""
    x = dev(kinds_of_rows(np.random.default_rng(vocab), vocab), dtype)
    for k in (129, 600, 1025, 2049, 5000, vocab // 2, vocab - 1):
        k = np.full(9, k, np.int32)
        check(pp.token_probs(x, top_k=dev(k)), x, None, k)
    biggest = torch.finfo(dtype).max
    x[0, ::3], x[0, 1::3] = biggest, -biggest  # further apart than a float
    x[8, 5] = biggest
    k = np.full(9, vocab // 2 + 1, np.int32)
    check(pp.token_probs(x, top_k=dev(k), temperature=dev(np.full(9, 1e30, np.float32))), x, np.full(9, 1e30), k)


@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 147461), (torch.float32, 262144), (torch.float16, 294919), (torch.bfloat16, 510007)])
def test_probs_of_the_longest_cuts(dtype, vocab):
    """Rows that only eight of the largest blocks hold, at any alignment."""
    there, _ = placed(9, vocab, dtype, vocab + 3, 1)
    there.copy_(dev(kinds_of_rows(np.random.default_rng(vocab), vocab), dtype))
    for k in (1, 50, 1500, 5000, vocab - 1):
        k = np.full(9, k, np.int32)
        check(pp.token_probs(there, top_k=dev(k)), there, None, k)
    t = np.array([0, 0.5, 1, 2, 0, 0.1, 1, 1, 1], np.float32)
    k = np.array([3, 0, -1, vocab, 0, 7, vocab + 1, 4096, 4097], np.int32)
    check(pp.token_probs(there, temperature=dev(t), top_k=dev(k)), there, t, k)


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("vocab", [50001, 82003, 101001, 120007, 180011, 210001])
def test_probs_in_clusters_of_any_size(dtype, vocab):
    """From two blocks a row to eight."""
    rng = np.random.default_rng(vocab)
    x = dev(kinds_of_rows(rng, vocab)[rng.integers(0, 9, 46)], dtype)
    k = np.exp(rng.uniform(0, np.log(vocab), 46)).astype(np.int32)
    k[::9] = 0
    t = rng.uniform(0.2, 3, 46).astype(np.float32)
    t[::17] = 0
    check(pp.token_probs(x, temperature=dev(t), top_k=dev(k)), x, t, k)
    check(pp.token_probs(x, temperature=dev(t)), x, t)


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("rows,vocab", [(3, 33000), (300, 9001), (2, 131075), (610, 1027), (2, 160000)])
def test_probs_into_rows_that_lie_otherwise(dtype, rows, vocab):
    """Results whose 16-byte boundaries are not the logits'."""
    rng = np.random.default_rng(rows)
    x = logits(rng, rows, vocab, dtype)
    k = np.exp(rng.uniform(0, np.log(vocab), rows)).astype(np.int32)
    t = rng.uniform(0.3, 2.0, rows).astype(np.float32)
    t[::5] = 0
    for cut in (None, k):
        out, whole = placed(rows, vocab, torch.float32, vocab + 5, 3)
        pp.token_probs(x, temperature=dev(t), top_k=None if cut is None else dev(cut), out=out)
        assert torch.equal(out, pp.token_probs(x, temperature=dev(t), top_k=None if cut is None else dev(cut)))
        check(out, x, t, cut)
        there = torch.zeros_like(whole, dtype=torch.bool)
        torch.as_strided(there, (rows, vocab), (vocab + 5, 1), 3).fill_(True)
        assert (whole[~there] == 77).all()


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("rows,vocab", [(609, 257), (610, 1027), (611, 4600), (1215, 33)])
def test_probs_of_many_short_rows(dtype, rows, vocab):
    """Several rows a block, the last of which has fewer; every length of a cut at once."""
    rng = np.random.default_rng(rows)
    kinds = kinds_of_rows(rng, vocab)
    x = kinds[rng.integers(0, 9, rows)] + 0.0
    x[::2] = rng.normal(0, 2, x[::2].shape)
    x = dev(x, dtype)
    k = rng.integers(0, vocab + 2, rows).astype(np.int32)
    k[::3] = np.minimum(k[::3], 5)
    t = rng.uniform(0.2, 3, rows).astype(np.float32)
    t[::17] = 0
    check(pp.token_probs(x, temperature=dev(t), top_k=dev(k)), x, t, k)
    check(pp.token_probs(x, temperature=dev(t)), x, t)
    again = x.float().clone()
    want = pp.token_probs(again, top_k=dev(k))
    assert torch.equal(pp.token_probs(again, top_k=dev(k), out=again), want)


def test_probs_has_no_derivative():
    x = torch.randn(2, 50, device="cuda", requires_grad=True)
    y = pp.token_probs(x)
    assert torch.equal(y, pp.token_probs(x.detach()))
    with pytest.raises(RuntimeError, match="token_probs has no derivative"):
        y.sum().backward()
    with torch.no_grad():
        assert not pp.token_probs(x).requires_grad


# ------------------------------------------------------------ verification
def drafted(rng, n, k, vocab, ragged, dtype=torch.float32):
    """Target's and drafts' rows behind one another, tokens drawn from the drafts' rows."""
    size = rng.integers(0, k + 1, n) if ragged else np.full(n, k)
    at = np.concatenate([[0], np.cumsum(size + 1)[:-1]])
    qat = np.concatenate([[0], np.cumsum(size)[:-1]])

    def soft(x):
        e = np.exp(x - x.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)

    z = rng.normal(0, 2, (int(size.sum()) + n, vocab))
    own = np.concatenate([np.arange(a, a + s) for a, s in zip(at, size)]).astype(int)
    p = dev(soft(z), torch.float32).to(dtype)
    q = dev(soft(z[own] + rng.normal(0, 0.7, (len(own), vocab))) if len(own) else np.zeros((0, vocab)), torch.float32).to(dtype)
    drafts = np.full((n, k), -1, np.int64)
    hq = wide(q)
    for r in range(n):
        for i in range(size[r]):
            drafts[r, i] = rng.choice(vocab, p=hq[qat[r] + i] / hq[qat[r] + i].sum())
    return dict(target=p, draft_probs=q, drafts=drafts, lengths=size.astype(np.int32), target_row=at.astype(np.int32),
                draft_row=qat.astype(np.int32), accept=rng.random((n, k)).astype(np.float32),
                sample=rng.random(n).astype(np.float32))


def run(a, **kw):
    a = dict(a, **kw)
    itype = a.pop("itype", torch.int32)
    args = {key: v if isinstance(v, torch.Tensor) or v is None else dev(v) for key, v in a.items()}
    args["drafts"] = args["drafts"].to(itype)
    ref = {key: wide(v) if isinstance(v, torch.Tensor) else v for key, v in a.items()}
    tokens, counts = pp.verify_drafts(**args)
    want, many = R.verify(**ref)
    assert tokens.dtype == counts.dtype == torch.int32
    assert np.array_equal(tokens.cpu().numpy(), want), (tokens.cpu().numpy() != want).any(1).nonzero()
    assert np.array_equal(counts.cpu().numpy(), many)
    return want, many


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("n,k,vocab,ragged", [(1, 0, 1, False), (1, 1, 2, False), (3, 4, 31, True), (7, 3, 100, False),
                                              (5, 40, 33, True), (2, 5, 5003, False), (33, 2, 4097, True), (2, 3, 70001, True),
                                              (1, 2, 131072, False), (400, 1, 300, True), (650, 3, 40, True)])
def test_verify(dtype, n, k, vocab, ragged):
    a = drafted(np.random.default_rng(n * 100 + k), n, k, vocab, ragged, dtype)
    run(a)
    run(a, draft_probs=None, draft_row=None)
    if not ragged:  # rows where they lie without lists
        run(a, target_row=None, draft_row=None, lengths=None)


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("vocab", [1, 2, 64, 65, 32768, 32769, 65536, 65537])
def test_verify_of_the_largest_sums(dtype, vocab):
    """All weights 1: sums up to 2^62 units, on both sides of where a probability takes another digit."""
    p = torch.ones(8, vocab, device="cuda", dtype=dtype)
    sample = np.array([0, 0.25, 0.5, 0.999, 1 - 2.0 ** -24, 2.0 ** -31, 1e-9, 0.75], np.float32)
    run(dict(target=p, drafts=np.zeros((8, 0), int), accept=np.zeros((8, 0), np.float32), sample=sample))
    run(dict(target=p, drafts=np.zeros((4, 1), int), accept=np.array([[0.5], [0.99], [0.0], [1.0]], np.float32), sample=sample[:4]))


@pytest.mark.parametrize("itype", IT)
def test_verify_token_types(itype):
    a = drafted(np.random.default_rng(5), 20, 4, 120, True)
    run(a, itype=itype, drafts=np.where(a["drafts"] < 0, 0, a["drafts"]))


def test_verify_draws_what_the_target_says():
    """Over many requests with one target the first tokens follow its probabilities,
    whatever the draft's were.  A share of n draws is within 5 standard deviations."""
    rng = np.random.default_rng(6)
    n, vocab = 200000, 5
    p, q = np.array([0.4, 0.3, 0.05, 0.25, 0.0]), np.array([0.1, 0.1, 0.5, 0.1, 0.2])
    drafts = rng.choice(vocab, (n, 1), p=q).astype(np.int32)
    args = dict(target=dev(np.stack([p, p]).astype(np.float32)), drafts=dev(drafts), accept=dev(rng.random((n, 1)).astype(np.float32)),
                sample=dev(rng.random(n).astype(np.float32)), target_row=torch.zeros(n, dtype=torch.int32, device="cuda"))
    for more in (dict(draft_probs=dev(q[None].astype(np.float32)), draft_row=torch.zeros(n, dtype=torch.int32, device="cuda")),
                 dict(drafts=torch.zeros(n, 1, dtype=torch.int32, device="cuda"))):  # and with a draft that is always token 0
        tokens, _ = pp.verify_drafts(**dict(args, **more))
        share = np.bincount(tokens[:, 0].cpu().numpy(), minlength=vocab) / n
        assert (np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / n)).all(), share


def test_verify_of_bad_tokens_rows_and_numbers():
    rng = np.random.default_rng(7)
    a = drafted(rng, 24, 4, 50, False)
    d = a["drafts"].copy()
    d[0, 0], d[1, 1], d[2, 3], d[3, 0] = -1, 50, 2 ** 31 - 1, -2 ** 31
    u = a["accept"].copy()
    u[4, 0], u[5, 1], u[6, 0], u[7] = np.nan, -0.5, 0.0, 1.0
    s = a["sample"].copy()
    s[8:14] = [np.nan, -1.0, 1.0, 2.0, 0.0, np.float32(1 - 2.0 ** -24)]
    rows = a["target_row"].copy()
    rows[14:19] = [-1, 2 ** 31 - 1, 118, 117, -2 ** 31]
    qrows = a["draft_row"].copy()
    qrows[19:23] = [-2, 96, 2 ** 31 - 1, 94]
    size = a["lengths"].copy()
    size[20:24] = [-3, 9, 2 ** 31 - 1, 0]
    b = dict(a, drafts=d, accept=u, sample=s, target_row=rows, draft_row=qrows, lengths=size)
    run(b)
    run(b, draft_probs=None, draft_row=None)
    p = a["target"].clone()
    p[::3, ::5] = torch.nan
    p[1::3, ::7] = torch.inf
    p[2::3, ::4] = -0.5
    p[5] = 0
    q = a["draft_probs"].clone()
    q[::4, ::3] = torch.nan
    q[1::4] = 2.0
    q[2::4, 1::2] = -torch.inf
    run(b, target=p, draft_probs=q)
    run(b, target=torch.zeros_like(p))
    run(b, target=torch.ones_like(p))  # sums of what is no distribution
    run(a, target=torch.ones_like(p), draft_probs=torch.full_like(q, 1e-3))
    run(b, target=p[:0])
    run(a, draft_probs=a["target"][:96], target=a["target"])  # mostly others' rows


@pytest.mark.parametrize("vocab", [50, 9000])
def test_verify_when_the_draft_leaves_nothing(vocab):
    """The target's own probabilities then: p nowhere above q, and a sure draft that is all the target has."""
    rng = np.random.default_rng(8)
    a = drafted(rng, 6, 1, vocab, False)
    p = a["target"].clone()
    q = torch.minimum(p[::2] * 1.5, torch.ones((), device="cuda"))
    run(a, target=p, draft_probs=q, accept=np.full((6, 1), 0.999, np.float32))
    p[::2] = 0
    p[torch.arange(0, 12, 2), torch.from_numpy(a["drafts"][:, 0]).cuda()] = 0.5
    want, _ = run(a, target=p, draft_probs=None, draft_row=None, accept=np.full((6, 1), 0.9, np.float32))
    assert (want[:, 0] == a["drafts"][:, 0]).all()


def test_verify_strides_outputs_and_no_requests():
    rng = np.random.default_rng(9)
    a = drafted(rng, 9, 3, 205, False)
    t, _ = placed(36, 205, torch.float32, 211, 3)
    t.copy_(a["target"])
    q, _ = placed(27, 205, torch.float32, 209, 1)
    q.copy_(a["draft_probs"])
    d, _ = placed(9, 3, torch.int32, 5, 1)
    d.copy_(dev(a["drafts"]))
    u, _ = placed(9, 3, torch.float32, 4, 1)
    u.copy_(dev(a["accept"]))
    out, whole = placed(9, 4, torch.int32, 7, 2)
    counts = torch.zeros(9, dtype=torch.int32, device="cuda")
    got = pp.verify_drafts(t, d, u, dev(a["sample"]), draft_probs=q, out=(out, counts))
    assert got[0] is out and got[1] is counts
    want, many = R.verify(wide(t), a["drafts"], a["accept"], a["sample"], wide(q))
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(counts.cpu().numpy(), many)
    there = torch.zeros_like(whole, dtype=torch.bool)
    torch.as_strided(there, (9, 4), (7, 1), 2).fill_(True)
    assert (whole[~there] == 77).all()
    empty = pp.verify_drafts(t, d[:0], u[:0], torch.zeros(0, device="cuda"))
    assert empty[0].shape == (0, 4) and empty[1].shape == (0,)


def test_verify_past_32_bit_offsets():
    rows, vocab = 17000, 131072
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    p = torch.zeros(rows, vocab, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    p[-3:] = torch.softmax(torch.randn(3, vocab, device="cuda", generator=g) * 3, 1)
    q = torch.softmax(torch.randn(2, vocab, device="cuda", generator=g) * 3, 1)
    a = dict(drafts=np.array([[5, 9]]), accept=np.array([[0.999, 0.5]], np.float32), sample=np.array([0.7], np.float32))
    tokens, counts = pp.verify_drafts(p, dev(a["drafts"]), dev(a["accept"]), dev(a["sample"]), draft_probs=q,
                                      target_row=torch.tensor([rows - 3], dtype=torch.int32, device="cuda"))
    want, many = R.verify(wide(p[-3:]), a["drafts"], a["accept"], a["sample"], wide(q))
    assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(counts.cpu().numpy(), many)


# ------------------------------------------------------------ streams, graphs, the run of them together
def test_other_streams_and_graphs():
    rng = np.random.default_rng(10)
    a = drafted(rng, 8, 3, 2003, True)
    x = logits(rng, 10, 2003, torch.bfloat16)
    k = dev(np.arange(10).astype(np.int32))
    args = dict({key: dev(v) if isinstance(v, np.ndarray) else v for key, v in a.items()})
    want_p, want_t = pp.token_probs(x, top_k=k), pp.verify_drafts(**args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [(pp.token_probs(x, top_k=k, stream=s), pp.verify_drafts(**args, stream=s)) for s in streams]
    torch.cuda.synchronize()
    for p, t in got:
        assert torch.equal(p, want_p) and torch.equal(t[0], want_t[0]) and torch.equal(t[1], want_t[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p = pp.token_probs(x, top_k=k)
        t = pp.verify_drafts(**args)
    other, more = logits(rng, 10, 2003, torch.bfloat16), rng.random(8).astype(np.float32)
    want_p = pp.token_probs(other, top_k=k)
    want_t = pp.verify_drafts(**dict(args, sample=dev(more)))
    x.copy_(other)
    args["sample"].copy_(dev(more))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p, want_p) and torch.equal(t[0], want_t[0]) and torch.equal(t[1], want_t[1])


def test_a_drafted_answer_keeps_to_the_grammar():
    """As they are used together: drafts' states from the grammar, masked logits of all
    positions, their probabilities, what is accepted, and the states after it."""
    words = [b"<end>", b",", b"\n", b'"', b"name", b"12.5", b"x y", b"q"]
    data = b"".join(b'"' + w.replace(b'"', b'""') + b'"\n' for w in words)
    (column,), _ = pp.parse_csv(torch.frombuffer(bytearray(data), dtype=torch.uint8).cuda(), ["str"])
    g = pp.vocab_grammar(*column, pp.desc_csv(), end_id=0)
    rng = np.random.default_rng(11)
    n, k, vocab = 500, 4, len(words)
    drafts = dev(rng.integers(0, vocab, (n, k)).astype(np.int32))
    before = pp.grammar_states(g, drafts)  # the state before each draft, and after the last
    raw = dev(rng.normal(0, 2, (n * (k + 1), vocab)), torch.float32)
    masked = pp.process_logits(raw, grammar=g, states=before.reshape(-1))
    target = pp.token_probs(masked, top_k=torch.full((n * (k + 1),), 5, dtype=torch.int32, device="cuda"))
    accept, sample = dev(rng.random((n, k)).astype(np.float32)), dev(rng.random(n).astype(np.float32))
    tokens, counts = pp.verify_drafts(target, drafts, accept, sample)
    ref, _ = R.probs(wide(masked), None, np.full(n * (k + 1), 5))
    want, many = R.verify(wide(target), drafts.cpu().numpy(), wide(accept), wide(sample))
    assert np.allclose(wide(target), ref, atol=1e-6)
    assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(counts.cpu().numpy(), many)
    after = pp.grammar_states(g, tokens, lengths=counts)
    # a sure draft that is any of the tokens alike is accepted with the mean of p, an eighth; 5 deviations of 500 draws
    assert abs((counts > 1).float().mean().item() - 1 / 8) < 5 * np.sqrt(1 / 8 * 7 / 8 / n)
    accepted = counts.cpu().numpy()
    ends = after.cpu().numpy()[np.arange(n), accepted]
    dead = (after == 4).any(1).cpu().numpy()  # the CSV DFA's invalid state
    assert not dead.any() and (ends != 255).all()
    # a state that allows nothing: no token
    none = pp.token_probs(pp.process_logits(raw[:1], grammar=g, states=torch.tensor([255], dtype=torch.uint8, device="cuda")))
    t, c = pp.verify_drafts(none, drafts[:1, :0], accept[:1, :0], sample[:1])
    assert t.tolist() == [[-1]] and c.tolist() == [0]


@pytest.mark.parametrize("seed,drafted", [(1, 3), (2, 1), (3, 0), (4, 7)])
def test_the_example_answers_what_parses_however_much_is_drafted(seed, drafted):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "grammar_rows.py")
    spec = importlib.util.spec_from_file_location("grammar_rows", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    out = example.run(seed=seed, drafted=drafted)
    assert out["same_states"] and out["said"] > 0 and out["rounds"] <= 48
    done = [p for p in out["parsed"] if p is not None]
    assert all(p["error"] & pp.ERR_FATAL == 0 for p in done)
    assert all(p is not None for p, over in zip(out["parsed"], out["over"]) if over)
