"""embed and embed_grad under torch's autograd: each is linear in its values
and the other one is its derivative, of any order."""
import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp


def plain_embed(ids, table, scale, padding_id, out=None, dtype=None, stream=None):
    """The kernels' results by torch on the CPU, cut from its graph as theirs are."""
    table = table.detach()
    there = (ids >= 0) & (ids < table.size(0)) & (ids != (-1 if padding_id is None else padding_id))
    rows = table[torch.where(there, ids, 0)] * scale
    return torch.where(there[..., None], rows, 0.0).to(table.dtype if dtype is None else dtype)


def plain_embed_grad(ids, grad, n_vocab, scale=1.0, padding_id=None, out=None, accumulate=False, dtype=None, stream=None):
    grad, ids = grad.detach().reshape(-1, grad.size(-1)), ids.flatten()
    there = (ids >= 0) & (ids < n_vocab) & (ids != (-1 if padding_id is None else padding_id))
    full = torch.zeros(n_vocab, grad.size(-1), dtype=grad.dtype).index_add_(0, ids[there], grad[there])
    return (full * scale).to(grad.dtype if dtype is None else dtype)


@pytest.fixture
def on_cpu(monkeypatch):
    """The two kernel calls replaced: what is tested is what autograd makes of them."""
    monkeypatch.setattr(pp.lm, "_embed", plain_embed)
    monkeypatch.setattr(pp.lm, "_embed_grad", plain_embed_grad, raising=False)


IDS = torch.tensor([[3, 0, 3], [6, -1, 2], [3, 9, 6]])  # 2: padding; -1 and 9: outside


def of(table):
    return pp.embed(IDS, table, scale=1.5, padding_id=2)


def test_derivatives_of_embed(on_cpu):
    table = torch.randn(7, 5, dtype=torch.float64, requires_grad=True)
    assert torch.autograd.gradcheck(of, (table,))
    assert torch.autograd.gradgradcheck(lambda t: of(t) ** 2, (table,))


def test_derivatives_of_embed_grad(on_cpu):
    grad = torch.randn(3, 3, 5, dtype=torch.float64, requires_grad=True)

    def f(g):
        return pp.embed_grad(IDS, g, 7, scale=1.5, padding_id=2)

    assert f(grad).requires_grad
    assert torch.autograd.gradcheck(f, (grad,))
    assert torch.autograd.gradgradcheck(lambda g: f(g) ** 2, (grad,))
    with torch.no_grad():
        assert not f(grad).requires_grad


def test_refuses_a_result_tensor_for_a_gradient_that_requires_one():
    grad = torch.zeros(4, 8, requires_grad=True)
    with pytest.raises(ValueError, match="out"):
        pp.embed_grad(torch.zeros(4, dtype=torch.int64), grad, 9, out=torch.zeros(9, 8))


def penalised(table, ids, weight, look_up):
    """A loss with the square of its own gradient, all in whole numbers."""
    y = look_up(ids, table)
    g, = torch.autograd.grad((weight * y * y).sum(), table, create_graph=True)
    return (weight * y).sum() + (g * g).sum()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [30, 2000])  # one kernel, and three
def test_gradient_penalty(n):
    rng = np.random.default_rng(n)
    vocab, dim = 40, 12
    ids = torch.from_numpy(rng.integers(-1, vocab + 1, (n // 10, 10)))
    value = torch.from_numpy(rng.integers(-3, 4, (vocab, dim))).double()
    weight = torch.from_numpy(rng.integers(0, 2, (*ids.shape, dim))).double()

    def plain(ids, table):
        there = (ids >= 0) & (ids < vocab) & (ids != 5)
        return torch.where(there[..., None], 2 * table[torch.where(there, ids, 0)], 0.0)

    host = value.clone().requires_grad_()
    penalised(host, ids, weight, plain).backward()
    table = value.float().cuda().requires_grad_()
    loss = penalised(table, ids.cuda(), weight.float().cuda(), lambda i, t: pp.embed(i, t, scale=2.0, padding_id=5))
    loss.backward()
    assert host.grad.abs().max() < 2 ** 24  # so that 32 bits hold every sum
    assert torch.equal(table.grad.double().cpu(), host.grad)


def test_forward_mode(on_cpu):
    """A dual tensor does not require a gradient, and still has a tangent."""
    import torch.autograd.forward_ad as forward
    table, tangent = torch.randn(2, 7, 5, dtype=torch.float64)
    grad, other = torch.randn(2, 3, 3, 5, dtype=torch.float64)
    with forward.dual_level():
        got = forward.unpack_dual(of(forward.make_dual(table, tangent))).tangent
        assert got is not None and torch.equal(got, of(tangent))
        dual = forward.make_dual(grad, other)
        got = forward.unpack_dual(pp.embed_grad(IDS, dual, 7, scale=1.5, padding_id=2)).tangent
        assert got is not None and torch.equal(got, pp.embed_grad(IDS, other, 7, scale=1.5, padding_id=2))
        with pytest.raises(ValueError, match="out"):
            pp.embed(IDS, forward.make_dual(table, tangent), out=torch.zeros(3, 3, 5, dtype=torch.float64))
        with pytest.raises(ValueError, match="out"):
            pp.embed_grad(IDS, dual, 7, out=torch.zeros(7, 5, dtype=torch.float64))
    table.requires_grad_()
    assert torch.autograd.gradcheck(of, (table,), check_forward_ad=True)
    assert torch.autograd.gradgradcheck(lambda t: of(t) ** 2, (table,), check_fwd_over_rev=True)


@pytest.mark.gpu
def test_forward_mode_of_the_kernels():
    import torch.autograd.forward_ad as forward
    rng = np.random.default_rng(1)
    table, tangent = torch.from_numpy(rng.integers(-9, 10, (2, 40, 12))).float().cuda()
    ids = torch.from_numpy(rng.integers(-1, 41, 100)).cuda()
    with forward.dual_level():
        y = pp.embed(ids, forward.make_dual(table, tangent), scale=2.0)
        d = pp.embed_grad(ids, y, 40, scale=0.5)
        value, slope = forward.unpack_dual(d)
    assert torch.equal(value, pp.embed_grad(ids, pp.embed(ids, table, scale=2.0), 40, scale=0.5))
    assert torch.equal(slope, pp.embed_grad(ids, pp.embed(ids, tangent, scale=2.0), 40, scale=0.5))


FLOATS = ["logits", "repetition", "presence", "frequency", "bias"]


def logit_arguments(device, follow=lambda t: t, which=None):
    f = {"logits": torch.ones(2, 9, device=device), "repetition": torch.ones(2, device=device),
         "presence": torch.ones(2, device=device), "frequency": torch.ones(2, device=device),
         "bias": torch.ones(2, device=device)}
    if which is not None:
        f[which] = follow(f[which])
    at = torch.tensor([0, 1, 2], dtype=torch.int32, device=device)
    f["bias"] = (at, at[:2], f["bias"])
    return dict(f, history=torch.zeros(2, 3, dtype=torch.int32, device=device))


@pytest.mark.parametrize("which", FLOATS)
def test_process_logits_has_no_derivative_and_says_so(monkeypatch, which):
    """Whoever differentiates its result is told; who does not, may go on."""
    import torch.autograd.forward_ad as forward
    monkeypatch.setattr(pp.lm, "_call", lambda *a: None)
    y = pp.process_logits(**logit_arguments("cpu", lambda t: t.requires_grad_(), which))
    assert y.requires_grad and y.argmax(1).shape == (2,)
    with pytest.raises(RuntimeError, match="process_logits"):
        (y.sum() + 1).backward()
    with pytest.raises(ValueError, match="out"):
        pp.process_logits(**logit_arguments("cpu", lambda t: t.requires_grad_(), which), out=torch.zeros(2, 9))
    with torch.no_grad():
        y = pp.process_logits(**logit_arguments("cpu", lambda t: t.requires_grad_(), which), out=torch.zeros(2, 9))
        assert not y.requires_grad
    with forward.dual_level(), pytest.raises(RuntimeError, match="process_logits"):
        pp.process_logits(**logit_arguments("cpu", lambda t: forward.make_dual(t, t), which))
    with forward.dual_level():
        assert not pp.process_logits(**logit_arguments("cpu")).requires_grad


@pytest.mark.gpu
def test_process_logits_of_logits_that_require_a_gradient():
    a = logit_arguments("cuda")
    want = pp.process_logits(**a)
    got = pp.process_logits(**dict(a, logits=a["logits"].clone().requires_grad_()))
    assert got.requires_grad and torch.equal(got.detach(), want)


def results(device):
    """Each operator with a result tensor: (its call, the shape and type of that)."""
    ids = torch.zeros(4, dtype=torch.int64, device=device)
    x = torch.zeros(4, 8, device=device)
    g = pp.Grammar(torch.zeros(9, dtype=torch.int64, device=device), torch.zeros(5, 4, dtype=torch.int32, device=device), 9,
                   pp.desc_csv())
    return {"grammar_states": (lambda out: pp.grammar_states(g, ids[None], out=out), (1, 5), torch.uint8),
            "process_logits": (lambda out: pp.process_logits(x, out=out), (4, 8), torch.float32),
            "embed": (lambda out: pp.embed(ids, x, out=out), (4, 8), torch.float32),
            "embed_grad": (lambda out: pp.embed_grad(ids, x, 9, out=out), (9, 8), torch.float32),
            "embed_grad added": (lambda out: pp.embed_grad(ids, x, 9, out=out, accumulate=True), (9, 8), torch.float32)}


def write_over_what_backward_needs(which, device):
    call, shape, dtype = results(device)[which]
    saved = torch.ones(shape, dtype=dtype, device=device)
    loss = (torch.ones(shape, device=device, requires_grad=True) * saved).sum()
    call(saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


RESULTS = ["grammar_states", "process_logits", "embed", "embed_grad", "embed_grad added"]


@pytest.mark.parametrize("which", RESULTS)
def test_results_in_place_are_noticed_by_autograd(monkeypatch, which):
    monkeypatch.setattr(pp.lm, "_call", lambda *a: None)
    write_over_what_backward_needs(which, "cpu")
    call, shape, dtype = results("cpu")[which]
    if dtype == torch.float32:
        leaf = torch.zeros(shape, requires_grad=True)
        with pytest.raises(ValueError, match="out"):
            call(leaf)
        with torch.no_grad():  # as a step of an optimiser may
            assert call(leaf) is leaf
    with torch.inference_mode():
        made = torch.zeros(shape, dtype=dtype)
        call(made)
    call(made)  # has no version to count


@pytest.mark.gpu
@pytest.mark.parametrize("which", RESULTS)
def test_results_in_place_on_the_gpu(which):
    write_over_what_backward_needs(which, "cuda")
    call, shape, dtype = results("cuda")[which]
    with torch.inference_mode():
        made = torch.zeros(shape, dtype=dtype, device="cuda")
        call(made)
    call(made)
