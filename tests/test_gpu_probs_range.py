"""GPU tests of probabilities far below a row's largest, wherever in the row and in
whatever blocks they are, and of the likeliest ones' last bits, against 64 bits."""
import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp

pytestmark = pytest.mark.gpu

FT = [torch.float32, torch.float16, torch.bfloat16]
U = 2.0 ** -24  # half a unit in the last place of 32 bits
# Additions on a term's way into its row's sum: a thread's values (9 vectors of 8), a warp's, a
# block's warps, a cluster's blocks.
ADDITIONS = 72 + 5 + 5 + 8
# What 32 bits hold below 2^-126 is off by a step of 2^-149 or two, in the exponential, in a
# block's factor and in their product.
LEAST = 2.0 ** -146


def formula(x, t, k=None):
    """(probabilities, distances y = (x - max) / t, the most that 32 bits may be off) in 64 bits.

    A value's exponent has four roundings: the difference, log2(e) / t twice, the product: 4 |y|
    u of the exponential; the exponential has 2 ulp, 4 u.  Where a block brings its values to
    the row's largest there are two such factors, whose distances add up to y: 8 u.  A sum of
    positive terms is off by what they are and by u for each addition on the way; the division
    and the product are u each, and the reciprocal of a reciprocal's place one more."""
    x, t = x.double(), torch.as_tensor(t, dtype=torch.float64, device=x.device).view(-1, 1)
    y = (x - x.max(1, keepdim=True).values) / t
    keep = torch.ones_like(x, dtype=torch.bool)
    if k is not None:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        rank = torch.empty_like(order).scatter_(1, order, torch.arange(x.size(1), device=x.device).expand_as(order))
        keep = rank < torch.where(k > 0, k, x.size(1))[:, None]
    keep &= x > -np.inf
    e = torch.where(keep, y.exp(), 0.0)
    z = e.sum(1, keepdim=True)
    term = (4 * torch.where(keep, -y, 0.0) + 8) * U
    of_sum = (e * term).sum(1, keepdim=True) / z + ADDITIONS * U
    p = e / z
    return p, y, p * (term + of_sum + 3 * U) + torch.where(keep, LEAST, 0.0)


def check(got, x, t, k=None):
    p, _, err = formula(x, t, k)
    off = (got.double() - p).abs()
    assert (off <= err).all(), ((off - err).max().item(), (off / p.clamp(min=1e-300)).max().item())


def numbers(n, value):
    return torch.full((n,), value, device="cuda")


# rows that two to eight blocks share, and short ones several of which share a block
SHAPES = [(1, 4100), (1, 32000), (5, 50001), (46, 50001), (46, 82003), (46, 101001), (3, 120007), (2, 131075), (610, 4000)]


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_far_parts_of_a_row(dtype, rows, vocab):
    """One logit far above the others, in each part of a row: the others' probabilities
    are small numbers that 32 bits hold."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    for peak in (40.0, 45.0, 55.0, 60.0, 66.0, 70.0, 80.0, 85.0):
        x = torch.randn(rows, vocab, generator=g, device="cuda").to(dtype)
        x[:, ::3] = 0.0  # equal logits in all parts
        at = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        x[torch.arange(rows, device="cuda"), at] = peak
        zero = torch.zeros(rows, dtype=torch.int32, device="cuda")
        check(pp.token_probs(x), x, 1.0)
        check(pp.token_probs(x, top_k=zero), x, 1.0)
        cool = x.float().mul(0.125).to(dtype)  # as far apart at a low temperature
        t = numbers(rows, 0.125)
        check(pp.token_probs(cool, temperature=t), cool, 0.125)
        check(pp.token_probs(cool, temperature=t, top_k=zero), cool, 0.125)


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("rows,vocab", [(1, 32000), (5, 50001), (3, 120007), (2, 131075), (3, 160000)])
def test_far_parts_of_a_cut_row(dtype, rows, vocab):
    """The same in cuts that the lists hold and in longer ones."""
    g = torch.Generator(device="cuda").manual_seed(vocab + 1)
    for peak in (40.0, 60.0, 80.0):
        x = torch.randn(rows, vocab, generator=g, device="cuda").to(dtype)
        x[:, vocab // 2] = peak
        for k in (50, 5000, vocab - 7):
            k = torch.full((rows,), k, dtype=torch.int32, device="cuda")
            got = pp.token_probs(x, top_k=k)
            check(got, x, 1.0, k)
            assert ((got > 0).sum(1) == k).all()


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("vocab", [9001, 32000, 50001])
def test_a_row_alone_and_among_others(dtype, vocab):
    """Shared out otherwise, a row keeps its probabilities."""
    g = torch.Generator(device="cuda").manual_seed(vocab + 2)
    row = torch.randn(1, vocab, generator=g, device="cuda").mul(3).to(dtype)
    row[0, vocab - 5] = 64.0
    row[0, 7::11] = -np.inf
    many = row.expand(1000, vocab).contiguous()
    for k in (None, 0, 600, vocab - 100):
        def cut(n):
            return None if k is None else torch.full((n,), k, dtype=torch.int32, device="cuda")
        alone, among = pp.token_probs(row, top_k=cut(1)), pp.token_probs(many, top_k=cut(1000))
        p, _, err = formula(row, 1.0, cut(1))
        assert ((alone.double() - p).abs() <= err).all()
        # (not the same bits: rows of an odd width begin at other places of a 16-byte vector, so other values meet in a thread)
        assert ((among.double() - p).abs() <= err).all()
        assert ((among > 0) == (alone > 0)).all()


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("rows,vocab", [(1, 32000), (700, 3001), (40, 50001), (300, 32000)])
def test_the_last_bits_of_likely_tokens(dtype, rows, vocab):
    """A probability over the largest's, in which the sum does not count: a factor e of
    (4 |y| + 8) u, a product and a quotient each on both sides, and what lies below 2^-126."""
    g = torch.Generator(device="cuda").manual_seed(vocab + 3)
    x = torch.rand(rows, vocab, generator=g, device="cuda").mul(-2.0).to(dtype)
    x[:, 11] = 0.0
    for k in (None, torch.zeros(rows, dtype=torch.int32, device="cuda")):
        got = pp.token_probs(x, top_k=k).double()
        _, y, _ = formula(x, 1.0)
        ratio = got / got[:, 11:12]
        assert ((ratio / y.exp() - 1).abs() <= (4 * -y + 8 + 3) * U * 1.01).all(), ((ratio / y.exp() - 1).abs() / U).max().item()


@pytest.mark.parametrize("dtype", FT)
def test_probabilities_that_are_subnormal(dtype):
    """Down to the least number above 0, in one block and in several."""
    x = torch.arange(0, 3000, device="cuda").mul(-0.04).to(dtype).repeat(700, 1)  # to 120 below
    check(pp.token_probs(x), x, 1.0)
    got = pp.token_probs(x[:1].repeat(1, 1), top_k=torch.zeros(1, dtype=torch.int32, device="cuda"))
    check(got, x[:1], 1.0)
    assert (got[0, :2440] > 0).all()  # 97.6 below, over a sum of 25.5: 2^-145.5
    wide = torch.cat([x[0], numbers(60000, -100.0).to(dtype)])[None]
    check(pp.token_probs(wide), wide, 1.0)


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("rows,vocab", [(1, 32000), (610, 4600), (9, 20011), (3, 131075), (2, 280003)])
def test_infinities_in_long_cuts(dtype, rows, vocab):
    """More infinities than the lists hold: the lowest of them share alike, in cuts that end
    among them and in cuts beyond."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=g, device="cuda").to(dtype)
    x[:, 3::2] = np.inf
    x[:, 5::7] = -np.inf
    many = int((x[0] == np.inf).sum())
    for k in (0, many - 100, many, many + 100, vocab // 4):
        got = pp.token_probs(x, top_k=torch.full((rows,), k, dtype=torch.int32, device="cuda"),
                             temperature=torch.full((rows,), 0.5, device="cuda"))
        keep = x == np.inf
        if 0 < k < many:
            keep &= torch.cumsum(keep, 1) <= k
        p = keep.double() / keep.sum(1, keepdim=True)
        assert ((got > 0) == keep).all() and ((got.double() - p).abs() <= 4 * U * p).all()
