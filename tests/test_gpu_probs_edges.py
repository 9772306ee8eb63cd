"""GPU tests of cuts that end exactly where a step of values ends, against plain
64-bit forms."""
import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp
import tokens_ref as R

pytestmark = pytest.mark.gpu

FT = [torch.float32, torch.float16, torch.bfloat16]
LEVELS = 100  # whole numbers 0 .. 99: exact in every type, and each in a step of its own of the 256


@pytest.mark.parametrize("dtype", FT)
@pytest.mark.parametrize("rows,vocab", [(3, 7001), (610, 4600), (200, 9000), (40, 20011), (46, 50001), (46, 82003), (46, 101001),
                                        (9, 131075), (5, 160000), (3, 280003)])
def test_cuts_that_end_at_a_steps_edge(dtype, rows, vocab):
    """All values of the last step are kept, so nothing is left to find among them; more
    than the lists of candidates hold, in blocks and clusters of every size."""
    rng = np.random.default_rng(vocab)
    x = rng.integers(0, LEVELS, (rows, vocab))
    k = np.zeros(rows, np.int32)
    for r in range(rows):
        run = np.cumsum(np.bincount(x[r], minlength=LEVELS)[::-1])
        at = np.flatnonzero(run > min(4096, vocab // 2))  # of lists with room for 4096 at most
        k[r] = run[at[rng.integers(0, len(at) - 1)]]
        if r % 5 == 4:
            k[r] += rng.integers(-1, 2)  # and one beside an edge
    there = torch.from_numpy(x.astype(np.float32)).cuda().to(dtype)
    t = np.full(rows, 30.0, np.float32)  # every kept token has a probability that is a float
    got = pp.token_probs(there, temperature=torch.from_numpy(t).cuda(), top_k=torch.from_numpy(k).cuda())
    ref, err = R.probs(x.astype(np.float64), t, k)
    got = got.double().cpu().numpy()
    assert np.array_equal(got > 0, ref > 0)
    assert (np.abs(got - ref) <= err).all()
