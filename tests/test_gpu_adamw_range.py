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


def changes(m, v, t, lr, betas, eps):
    """What parameters change by in 64 bits, and what they are off at most: 2^-19 of
    themselves, 2^-126, and 2^-126 over the divisor where the rate times the mean is less than that."""
    rate = np.float64(lr) / (1 - betas[0] ** t)
    below = np.sqrt(v / (1 - betas[1] ** t)) + np.float64(np.float32(eps))
    with np.errstate(divide="ignore", invalid="ignore"):
        change = np.where(m == 0, 0.0, rate * m / below)
        lost = np.where(np.abs(rate * m) < 2.0 ** -126, 2.0 ** -126 / below, 0.0)
    return change, 2.0 ** -19 * np.abs(change) + 2.0 ** -126 + np.where(m == 0, 0.0, lost)


def one_step(grad, lr, betas, eps, t=1):
    """(what parameters of 0 became, the states as 32 bits hold them)"""
    w = torch.zeros(grad.size, device="cuda")
    s = pp.adamw_state([w])
    s.step.fill_(t - 1)
    pp.adamw_step([w], [torch.from_numpy(grad).cuda()], s, lr=lr, betas=betas, eps=eps, weight_decay=0.0)
    m, v = wide(s.exp_avg)[:grad.size], wide(s.exp_avg_sq)[:grad.size]
    x, y = R.step32(np.zeros_like(grad), np.zeros_like(grad), grad.astype(np.float64), *betas)
    assert np.array_equal(m, x.astype(np.float64)) and np.array_equal(v, y.astype(np.float64))
    return wide(w), m, v


@pytest.mark.parametrize("beta2", [0.9, 0.99, 0.999, 0.9999, 0.999999])
@pytest.mark.parametrize("eps", [2.0 ** -41, 2.0 ** -40, 2.0 ** -39, 2.0 ** -36, 2.0 ** -31, 1e-8])
def test_subnormal_squares_beside_eps(eps, beta2):
    """The first step, whose 1 / sqrt(1 - beta2) makes the root of a square larger."""
    size = np.linspace(-64.0, -60.0, 1001) - 0.5 * np.log2(1 - beta2)
    grad = (2.0 ** size).astype(np.float32)
    grad[::2] *= -1
    got, m, v = one_step(grad, 1.0, (0.9, beta2), eps)
    assert v.min() < 2.0 ** -126 < v.max()
    change, most = changes(m, v, 1, 1.0, (0.9, beta2), eps)
    assert (np.abs(got + change) <= most).all(), (np.abs(got + change) / np.abs(change)).max()


@pytest.mark.parametrize("t", [1, 2, 50, 4000])
@pytest.mark.parametrize("eps", [1e-12, 2.0 ** -41, 1e-10, 1e-8, 1e-3])
@pytest.mark.parametrize("lr", [1e-3, 1.0, 1e-20])
def test_means_near_the_least_numbers(lr, eps, t):
    """Gradients from subnormal numbers up, of which the changes are what pp.h says."""
    size = np.linspace(-148.0, -20.0, 3001)
    grad = (2.0 ** size).astype(np.float32)
    grad[::2] *= -1
    got, m, v = one_step(grad, lr, (0.9, 0.999), eps, t)
    change, most = changes(m, v, t, lr, (0.9, 0.999), eps)
    assert (np.abs(got + change) <= most).all(), (np.abs(got + change) - most).max()
