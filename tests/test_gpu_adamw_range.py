"""GPU tests of the AdamW step where numbers of very different size meet, against plain
64-bit forms."""
import numpy as np
import pytest
import torch

import adamw_ref as R
import dfa_parsing_delimiter_gb300 as pp

pytestmark = pytest.mark.gpu


def wide(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("nearest", [True, False])
@pytest.mark.parametrize("top", [10, 15, 16, 17, 30, 45, 62, 63])
def test_a_small_square_beside_a_large_one_is_not_zero(top, nearest):
    """8-bit squares above 0 keep a code above 0, whatever the largest of their block: the
    step divides by their root."""
    n = 256 * 6 + 40  # whole tiles and the rest of one
    w = torch.zeros(n, device="cuda")
    s = pp.adamw_state([w], bits=8, seed=5, nearest=nearest)
    g = torch.Generator(device="cuda").manual_seed(top)
    # squares down to the least subnormal number, and zeros
    size = torch.randint(-74, 2, (n,), generator=g, device="cuda").double()
    grad = (2.0 ** size * torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, -1.0, 1.0)).float()
    grad[::7] = 0.0
    grad[::256] = 2.0 ** top
    grad[1::256] = -2.0 ** -30
    pp.adamw_step([w], [grad], s, betas=(0.5, 0.5), lr=1e-3)
    x, y = R.step32(np.zeros(n, np.float32), np.zeros(n, np.float32), wide(grad), 0.5, 0.5)
    r = (None, None) if nearest else R.dither(0, n, 5, 1)
    for got, e, z, rr, signed in ((s.exp_avg, s.exp_avg_exponent, x, r[0], True), (s.exp_avg_sq, s.exp_avg_sq_exponent, y, r[1], False)):
        c, ex = R.encode(z, rr, signed)
        assert np.array_equal(e.cpu().numpy(), ex)
        assert np.array_equal(got[:n].cpu().numpy(), c)
    assert ((s.exp_avg_sq[:n].cpu().numpy() > 0) == (y > 0)).all()
    before = w.clone()
    pp.adamw_step([w], [torch.zeros_like(grad)], s, betas=(0.5, 0.5), lr=1e-3)
    assert torch.isfinite(w).all() and ((w - before).abs() <= 1.0).all()
