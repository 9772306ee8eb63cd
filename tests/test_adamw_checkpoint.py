"""A training with 8-bit states that is saved and resumed rounds on as it would have."""
import io

import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp


def saved(state):
    f = io.BytesIO()
    torch.save(state.state_dict(), f)
    f.seek(0)
    return torch.load(f, weights_only=True)


@pytest.mark.parametrize("seed,nearest", [(7, False), (-1, False), (2 ** 32 + 5, False), (0, True)])
def test_how_states_are_rounded_is_saved(seed, nearest):
    w = [torch.randn(300), torch.randn(7)]
    s, t = pp.adamw_state(w, bits=8, seed=seed, nearest=nearest), pp.adamw_state(w, bits=8, seed=1, nearest=not nearest)
    d = saved(s)
    assert d["seed"].dtype == torch.int64 and d["nearest"].dtype == torch.bool
    t.load(**d)
    assert t.seed == s.seed == seed & 0xFFFFFFFF and t.nearest is nearest
    t.load(step=s.step)  # what is not given stays
    assert t.seed == s.seed and t.nearest is nearest
    for bad in (dict(seed=torch.tensor(1.0)), dict(seed=torch.zeros(2, dtype=torch.int64)), dict(nearest=torch.tensor(1))):
        with pytest.raises(ValueError):
            t.load(**bad)
    assert t.seed == s.seed


def test_states_of_32_bits_have_no_rounding():
    w = [torch.randn(300)]
    s = pp.adamw_state(w, seed=3)
    assert sorted(s.state_dict()) == ["exp_avg", "exp_avg_sq", "step"]
    with pytest.raises(ValueError):
        s.load(seed=torch.tensor(3))
    with pytest.raises(ValueError):  # states of another size of codes
        s.load(**pp.adamw_state(w, bits=8).state_dict())


@pytest.mark.gpu
@pytest.mark.parametrize("seed,nearest", [(7, False), (0, True)])
def test_a_resumed_training_has_the_same_bits(seed, nearest):
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(1000, device="cuda", generator=g)
    grads = [torch.randn(1000, device="cuda", generator=g) for _ in range(6)]
    a = w.clone()
    s = pp.adamw_state([a], bits=8, seed=seed, nearest=nearest)
    for x in grads[:3]:
        pp.adamw_step([a], [x], s)
    b, d = a.clone(), saved(s)
    t = pp.adamw_state([b], bits=8, seed=seed + 1)
    t.load(**d)
    for x in grads[3:]:
        pp.adamw_step([a], [x], s)
        pp.adamw_step([b], [x], t)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(s.state_dict().values(), t.state_dict().values()))
