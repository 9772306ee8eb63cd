"""Bias lists in which tokens are repeated: the last entry of each counts, at
a cost that grows with the list alone."""
import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp
import lm_ref as R
from test_gpu_lm import FT, dev, logit_case, on_gpu, random_grammar

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("hist", [None, 30, 70000])
@pytest.mark.parametrize("n", [2, 3, 33, 511, 512, 513, 1024, 1025, 3000])
def test_repeated_tokens(n, hist, dtype):
    """Within one lot of entries, across lots, in every row's own way."""
    rng = np.random.default_rng(n)
    rows, vocab = 6, 2051
    x, c = logit_case(rng, rows, vocab, dtype, hist=hist, n_bias=None)
    pool = [rng.integers(0, vocab, n),                                          # few pairs
            rng.integers(0, 3, n),                                              # nearly all the same
            np.concatenate([rng.permutation(vocab), rng.permutation(vocab)])[:n],  # pairs lots apart
            np.repeat(rng.integers(0, vocab, n), 2)[:n],                        # pairs side by side
            np.where(rng.random(n) < 0.5, -1, rng.integers(0, vocab + 50, n)),  # many outside
            np.full(n, 7)]
    at = (np.arange(rows + 1) * n).astype(np.int32)
    c["bias"] = (at, np.concatenate(pool).astype(np.int32), rng.normal(0, 5, rows * n).astype(np.float32))
    ref, error = R.logits(x.double().numpy(), **c)
    R.check(pp.process_logits(x.cuda(), **on_gpu(c)), ref, error, dtype)
    g, fine = random_grammar(rng, vocab)
    states = np.array([0, 1, 2, 3, 4, 2], np.uint8)
    ref, error = R.logits(x.double().numpy(), fine=fine[states], **c)
    got = x.cuda()
    pp.process_logits(got, grammar=g, states=dev(states), out=got, **on_gpu(c))  # in place
    R.check(got, ref, error, dtype)


def test_one_pair_in_a_long_list_costs_little():
    """A list of 100000 entries with one repeated token against the same
    without: each entry searched what follows it once one was repeated, 1000
    times the time.  Bounded here by 20 times."""
    n, vocab = 100000, 131072
    rng = np.random.default_rng(1)
    tokens = rng.permutation(vocab)[:n].astype(np.int32)
    at, values, x = dev(np.array([0, n], np.int32)), dev(np.ones(n, np.float32)), torch.zeros(1, vocab, device="cuda")

    def best(tokens):
        bias, times = (at, dev(tokens), values), []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            pp.process_logits(x, bias=bias)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times[1:])

    alone = best(tokens)
    tokens[n // 2] = tokens[10]
    assert best(tokens) < 20 * alone
