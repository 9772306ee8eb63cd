"""GPU tests of the AdamW step against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import adamw_ref as R
import dfa_parsing_delimiter_gb300 as pp

pytestmark = pytest.mark.gpu

FT = [torch.float32, torch.float16, torch.bfloat16]
# a rounding to the type: half a step, and half the least subnormal number
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -134)}
B1, B2, EPS = 0.9, 0.999, 1e-8
SHAPES = [(1,), (7,), (256,), (257,), (33, 67), (4, 2, 64), (0, 5), (5000,), ()]


def wide(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, err, dtype, what):
    rel, least = ROUND[dtype]
    bound = err + (rel * (np.abs(ref) + err) + least if dtype != torch.float32 else 0)
    off = np.abs(wide(got).ravel() - ref.ravel())
    assert (off <= bound.ravel()).all(), (what, (off - bound.ravel()).max())


class Model:
    """Tensors, their gradients and a state from the middle of a training."""

    def __init__(self, seed, shapes=SHAPES, dtype=torch.float32, gtype=torch.float32, bits=32, master=False, nearest=False, offset=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.params = [self.normal(s, 0.05, dtype, offset) for s in shapes]
        self.grads = [self.normal(s, 0.3, gtype, offset) for s in shapes]
        self.state = s = pp.adamw_state(self.params, bits=bits, master=master, seed=seed, nearest=nearest)
        s.step.fill_(10)
        m = torch.randn(s.n, device="cuda", generator=self.g) * 0.1
        v = (torch.randn(s.n, device="cuda", generator=self.g) * 0.1) ** 2
        inside = torch.zeros(s.n, dtype=torch.bool, device="cuda")
        for part in s.split(inside):
            part.fill_(True)
        m, v = torch.where(inside, m, 0.0), torch.where(inside, v, 0.0)
        if bits == 32:
            s.load(exp_avg=m, exp_avg_sq=v)
        else:
            for name, x, signed in (("exp_avg", m, True), ("exp_avg_sq", v, False)):
                c, e = R.encode(x.cpu().numpy(), None, signed)
                s.load(**{name: torch.from_numpy(c).cuda(), name + "_exponent": torch.from_numpy(e).cuda()})
        if master:
            for part, p in zip(s.split(s.master), self.params):
                part.mul_(1 + 1e-3 * torch.randn(part.shape, device="cuda", generator=self.g))

    def normal(self, shape, scale, dtype, offset=0):
        n = int(np.prod(shape))
        whole = torch.randn(n + offset, device="cuda", generator=self.g).mul_(scale).to(dtype)
        return whole[offset:].view(shape)

    def numbers(self):
        """(exp_avg, exp_avg_sq) in 64 bits."""
        s = self.state
        if s.bits == 32:
            return wide(s.exp_avg), wide(s.exp_avg_sq)
        return tuple(R.value(c.cpu().numpy(), e.cpu().numpy(), signed) for c, e, signed in (
            (s.exp_avg, s.exp_avg_exponent, True), (s.exp_avg_sq, s.exp_avg_sq_exponent, False)))

    def step_and_check(self, lr=1e-2, decay=0.1, scale=1.0, betas=(B1, B2), eps=EPS, **kw):
        s = self.state
        t = int(s.step) + 1
        m0, v0 = self.numbers()
        before = [wide(p) for p in (self.params if s.master is None else s.split(s.master))]
        decays = [decay] * len(self.params) if isinstance(decay, float) else decay
        pp.adamw_step(self.params, self.grads, s, lr=lr, betas=betas, eps=eps, weight_decay=decay, **kw)
        assert int(s.step) == t and s._counters.tolist() == [t, 0]
        if s.bits == 32:
            m1, v1 = s.exp_avg.cpu().numpy(), s.exp_avg_sq.cpu().numpy()
        for i, (a, n) in enumerate(zip(s.first, s.sizes)):
            if not n or self.grads[i] is None:
                continue
            g, m, v = wide(self.grads[i]).ravel(), m0[a:a + n], v0[a:a + n]
            # the factors as 32 bits hold them, as the formula's
            (p, m2, v2), (ep, em, ev) = R.step(before[i].ravel(), g, m, v, t, lr, betas[0], betas[1], eps, decays[i], scale)
            if s.master is not None:
                near(s.split(s.master)[i], p, ep, torch.float32, "master")
            near(self.params[i], p, ep, self.params[i].dtype, "param")
            x, y = R.step32(m.astype(np.float32), v.astype(np.float32), g, betas[0], betas[1], scale)
            assert (np.abs(x - m2) <= em).all() and (np.abs(y - v2) <= ev).all()
            if s.bits == 32:
                assert np.array_equal(m1[a:a + n], x) and np.array_equal(v1[a:a + n], y)
            else:
                r = (None, None) if s.nearest else R.dither(a, n, s.seed, t)
                b = -(-n // 256)
                for got, e, z, rr, signed in ((s.exp_avg, s.exp_avg_exponent, x, r[0], True),
                                              (s.exp_avg_sq, s.exp_avg_sq_exponent, y, r[1], False)):
                    c, ex = R.encode(z, rr, signed)
                    assert np.array_equal(e[a // 256:a // 256 + b].cpu().numpy(), ex)
                    assert np.array_equal(got[a:a + n].cpu().numpy(), c)
        for flat in (s.exp_avg, s.exp_avg_sq):  # what no tensor has stays 0
            outside = torch.ones(s.n, dtype=torch.bool, device="cuda")
            for part in s.split(outside):
                part.fill_(False)
            assert (flat[outside] == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,gtype,master", [(a, b, c) for a in FT for b in FT for c in (False, True)])
def test_steps(bits, dtype, gtype, master):
    m = Model(1, dtype=dtype, gtype=gtype, bits=bits, master=master)
    for _ in range(3):
        m.step_and_check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [1, 3, 4, 8])
@pytest.mark.parametrize("dtype", FT)
def test_unaligned_tensors(bits, offset, dtype):
    """Parameters and gradients at any element, and nothing beside them written."""
    m = Model(2, shapes=[(256,), (1000,), (513,), (3,)], dtype=dtype, gtype=dtype, bits=bits, offset=offset)
    before = [p._base[:offset].clone() for p in m.params]
    m.step_and_check()
    assert all(torch.equal(a, p._base[:offset]) for a, p in zip(before, m.params))


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zeros(bits):
    m = Model(3, bits=bits)
    s = m.state
    for x in s.state_dict().values():
        x.zero_()
    m.step_and_check()
    m.step_and_check(betas=(0.0, 0.0), decay=0.0)
    m.step_and_check(betas=(0.5, 0.0), decay=[0.0, 0.1, 0.2, 0.3, 0.4, 0.5, 0.6, 0.7, 0.8])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 2.0 ** -41, 2.0 ** -40, 1e-3])
def test_small_and_large_eps(bits, eps):
    """Also where a square is a subnormal number beside it."""
    m = Model(14, bits=bits)
    m.step_and_check(eps=eps)
    if bits == 32:  # (in 8 bits a block's largest decides)
        m.state.exp_avg.mul_(1e-16)
        m.state.exp_avg_sq.mul_(1e-36)
        for g in m.grads:
            g.mul_(1e-19)
        m.step_and_check(eps=eps, lr=1.0)


def test_many_steps_done():
    m = Model(4)
    m.state.step.fill_(2 ** 30)
    m.step_and_check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [16, 17, 128, 129, 640, 641, 1500])
def test_many_tensors(bits, count):
    """More than one launch takes, with empty ones between."""
    rng = np.random.default_rng(count)
    m = Model(5, shapes=[(int(n),) for n in rng.integers(0, 700, count)], bits=bits)
    m.step_and_check(decay=rng.uniform(0, 1, count).tolist())


@pytest.mark.parametrize("bits", [32, 8])
def test_large_tensor(bits):
    m = Model(6, shapes=[(3000, 1111), (5,)], gtype=torch.bfloat16, bits=bits)
    m.step_and_check()


@pytest.mark.parametrize("bits", [32, 8])
def test_left_out_gradients_and_none(bits):
    m = Model(7, shapes=[(300,), (300,), (40,)], bits=bits)
    m.grads[1] = None
    old = m.params[1].clone(), [m.state.split(x)[1].clone() for x in (m.state.exp_avg, m.state.exp_avg_sq)]
    m.step_and_check()
    assert torch.equal(m.params[1], old[0])
    assert all(torch.equal(m.state.split(x)[1], y) for x, y in zip((m.state.exp_avg, m.state.exp_avg_sq), old[1]))
    was = int(m.state.step)
    pp.adamw_step(m.params, [None] * 3, m.state)
    assert int(m.state.step) == was + 1 and torch.equal(m.params[1], old[0])


def test_leaves_and_their_own_gradients():
    w = torch.randn(40, 50, device="cuda", requires_grad=True)
    b = torch.randn(50, device="cuda", requires_grad=True)
    unused = torch.randn(3, device="cuda", requires_grad=True)
    s = pp.adamw_state([w, b, unused])
    x = torch.randn(9, 40, device="cuda")
    loss = ((x @ w + b) ** 2).sum()
    loss.backward(retain_graph=True)
    want = [R.step(wide(p), wide(p.grad), 0, 0, 1, 1e-3, B1, B2, EPS, 0.01) for p in (w, b)]
    pp.adamw_step([w, b, unused], None, s)
    for p, ((ref, _, _), (err, _, _)) in zip((w, b), want):
        near(p, ref, err, torch.float32, "param")
    assert w.requires_grad and w.is_leaf
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y = ((x @ w).exp() @ w.t()).sum()  # its backward pass needs w as it was
        pp.adamw_step([w, b, unused], None, s)
        y.backward()


@pytest.mark.parametrize("bits", [32, 8])
def test_numbers_on_the_device(bits):
    m = Model(8, bits=bits)
    scale = torch.tensor(0.25, device="cuda")
    lr = torch.tensor([0.02], device="cuda")
    m.step_and_check(scale=0.25, grad_scale=scale)
    before = wide(m.params[4])
    again = Model(8, bits=bits)
    pp.adamw_step(m.params, m.grads, m.state, lr=lr)
    assert not np.array_equal(before, wide(m.params[4]))
    pp.adamw_step(again.params, again.grads, again.state, lr=1e-2, weight_decay=0.1, grad_scale=scale)
    pp.adamw_step(again.params, again.grads, again.state, lr=float(lr))
    assert all(torch.equal(a, b) for a, b in zip(m.params, again.params))
    for flag in (1.0, float("nan"), float("inf"), -2.0):
        copy = [p.clone() for p in m.params], [x.clone() for x in m.state.state_dict().values()]
        m.grads[0].fill_(torch.nan)
        pp.adamw_step(m.params, m.grads, m.state, skip=torch.tensor(flag, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(copy[0], m.params))
        assert all(torch.equal(a, b) for a, b in zip(copy[1], m.state.state_dict().values()))
    m.grads[0].fill_(0.5)
    m.step_and_check(skip=torch.zeros((), device="cuda"))


def test_infinities_and_nan():
    """In 32 bits they stay where they are; in 8 bits the block that has one is NaN."""
    for bits in (32, 8):
        m = Model(9, shapes=[(1000,)], bits=bits)
        ref = Model(9, shapes=[(1000,)], bits=bits)
        m.grads[0][300], m.grads[0][700] = torch.nan, torch.inf
        for k in (m, ref):
            pp.adamw_step(k.params, k.grads, k.state)
        bad = torch.zeros(1000, dtype=torch.bool, device="cuda")
        bad[[300, 700]] = True
        assert torch.equal(m.params[0][~bad], ref.params[0][~bad]) and not torch.isfinite(m.params[0][300])
        for x, y in zip(m.state.values(), ref.state.values()):
            gone = bad if bits == 32 else ((torch.arange(1000, device="cuda") // 256 == 1) | (torch.arange(1000, device="cuda") // 256 == 2))
            assert torch.equal(x[:1000][~gone], y[:1000][~gone]) and not torch.isfinite(x[:1000][gone]).any()


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 3e18])
@pytest.mark.parametrize("bits", [32, 8])
def test_small_and_large_gradients(scale, bits):
    """Squares down to subnormal numbers and up to the largest."""
    m = Model(10, shapes=[(700,), (256,)], bits=bits, nearest=True)
    for x in m.state.state_dict().values():
        x.zero_()
    for g in m.grads:
        g.copy_(torch.randn(g.shape, device="cuda", generator=m.g) * scale)
    g = [wide(x).ravel().astype(np.float32) for x in m.grads]
    pp.adamw_step(m.params, m.grads, m.state, betas=(0.5, 0.5))
    for i, (a, n) in enumerate(zip(m.state.first, m.state.sizes)):
        with np.errstate(over="ignore"):
            x, y = R.step32(np.zeros(n, np.float32), np.zeros(n, np.float32), g[i], 0.5, 0.5)
        for got, z, signed in zip(m.state.values(), (x, y), (True, False)):
            want = z if bits == 32 else R.value(*R.encode(z, None, signed), signed)
            assert np.array_equal(wide(got)[a:a + n], want.astype(np.float32).astype(np.float64))
    assert all(torch.isfinite(p).all() for p in m.params)


def test_values_of_codes():
    """Every code under several exponents, in all types."""
    s = pp.adamw_state([torch.zeros(256 * 8, device="cuda")], bits=8)
    e = torch.tensor([0, 1, 2, 100, 127, 200, 253, 255], dtype=torch.uint8, device="cuda")
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(8)
    s.load(exp_avg=codes, exp_avg_sq=codes, exp_avg_exponent=e, exp_avg_sq_exponent=e)
    for dtype in FT:
        for got, signed in zip(s.values(dtype), (True, False)):
            want = torch.from_numpy(R.value(codes.cpu().numpy(), e.cpu().numpy(), signed)).float().to(dtype)
            assert torch.equal(got.cpu().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0)), dtype


def test_rounding_is_right_on_average():
    """Steps of v by 1/1000 of itself, smaller than half of any code's, arrive; and the two
    states' roundings have nothing to do with one another.  With n elements a mean of
    roundings between neighbours d apart is within 5 d / (2 sqrt(n)) of its own."""
    n = 1 << 20
    for seed in (0, 1, 12345):
        w = torch.zeros(n, device="cuda")
        s = pp.adamw_state([w], bits=8, seed=seed)
        g = torch.full((n,), 0.37, device="cuda")
        m = v = 0.0
        for t in range(40):
            pp.adamw_step([w], [g], s, lr=0.0)
            m, v = B1 * m + (1 - B1) * 0.37, B2 * v + (1 - B2) * 0.37 ** 2
            x, y = (k.double() for k in s.values())
            # neighbours are an eighth apart at most; errors of earlier steps add up, each once
            assert abs(float(x.mean()) / m - 1) < 5 * 0.125 / 2 / np.sqrt(n) * (t + 1) + 1e-4
            assert abs(float(y.mean()) / v - 1) < 5 * 0.125 / 2 / np.sqrt(n) * (t + 1) + 1e-4
        up, high = (x > x.mean()).double(), (y > y.mean()).double()
        for a, b in ((up, high), (up[1:], up[:-1]), (up[256:], up[:-256]), (high[1:], high[:-1])):
            a, b = a - a.mean(), b - b.mean()
            assert abs(float((a * b).mean() / (a.std() * b.std()))) < 5 / np.sqrt(n) + 1e-6
    # to nearest, from where it is: v stays, whatever it should be
    s = pp.adamw_state([w], bits=8, nearest=True)
    for _ in range(30):
        pp.adamw_step([w], [g], s, lr=0.0, betas=(B1, 0.0))
    at = s.values()[1].clone()
    for _ in range(30):
        pp.adamw_step([w], [g * 0], s, lr=0.0)
    assert torch.equal(at, s.values()[1])


def test_the_same_bits_again_and_another_seed():
    a, b, c = Model(11, bits=8), Model(11, bits=8), Model(11, bits=8)
    c.state.seed = 12
    for k in (a, b, c):
        for _ in range(5):
            pp.adamw_step(k.params, k.grads, k.state)
    assert all(torch.equal(x, y) for x, y in zip(a.state.state_dict().values(), b.state.state_dict().values()))
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
    assert not torch.equal(a.state.exp_avg_sq, c.state.exp_avg_sq)


@pytest.mark.parametrize("bits", [32, 8])
def test_streams_and_graphs(bits):
    """Captured and replayed, the step counts on and new gradients are read; other models
    step on other streams meanwhile."""
    a, b = Model(12, bits=bits), Model(12, bits=bits)
    g = torch.cuda.CUDAGraph()
    lr = torch.tensor(1e-2, device="cuda")
    with torch.cuda.graph(g):
        pp.adamw_step(a.params, a.grads, a.state, lr=lr)
    for k in range(4):
        for x, y in zip(a.grads, b.grads):
            y.copy_(torch.randn(y.shape, device="cuda", generator=b.g))
            x.copy_(y)
        lr.fill_(1e-2 / (k + 1))
        g.replay()
        pp.adamw_step(b.params, b.grads, b.state, lr=float(lr))
    assert int(a.state.step) == int(b.state.step) == 14
    assert all(torch.equal(x, y) for x, y in zip(a.params + list(a.state.state_dict().values()),
                                                 b.params + list(b.state.state_dict().values())))
    models = [Model(20 + k, bits=bits) for k in range(4)]
    same = [Model(20 + k, bits=bits) for k in range(4)]
    streams = [torch.cuda.Stream() for _ in models]
    torch.cuda.synchronize()
    for _ in range(3):
        for m, s in zip(models, streams):
            pp.adamw_step(m.params, m.grads, m.state, stream=s)
    torch.cuda.synchronize()
    for m in same:
        for _ in range(3):
            pp.adamw_step(m.params, m.grads, m.state)
    for m, n in zip(models, same):
        assert all(torch.equal(x, y) for x, y in zip(m.params, n.params)) and int(m.state.step) == 13


def test_parameters_from_an_iterator():
    """As torch.nn modules give them; and numbers that are no floats of Python's."""
    model = torch.nn.Sequential(torch.nn.Linear(7, 30), torch.nn.Linear(30, 2)).cuda()
    other = [p.detach().clone() for p in model.parameters()]
    a, b = pp.adamw_state(model.parameters()), pp.adamw_state(other)
    model(torch.ones(3, 7, device="cuda")).square().sum().backward()
    grads = [p.grad for p in model.parameters()]
    pp.adamw_step(model.parameters(), None, a, lr=0.1, weight_decay=np.float32(0.25))
    pp.adamw_step(iter(other), iter(grads), b, lr=np.float64(0.1), weight_decay=(0.25 for _ in grads))
    assert all(torch.equal(x, y) for x, y in zip(model.parameters(), other))
    assert [p._version for p in other] == [1] * 4


def test_master_copies_add_up_small_steps():
    """Steps of a hundredth of a bfloat16's: without 32-bit copies they are lost."""
    w = torch.ones(1000, dtype=torch.bfloat16, device="cuda")
    lost = w.clone()
    s, t = pp.adamw_state([w], master=True), pp.adamw_state([lost])
    g = torch.ones(1000, dtype=torch.bfloat16, device="cuda")
    for _ in range(300):
        pp.adamw_step([w], [g], s, lr=4e-5, weight_decay=0.0)
        pp.adamw_step([lost], [g], t, lr=4e-5, weight_decay=0.0)
    # Adam's first steps under one gradient are lr each: 300 of them
    assert abs(float(s.master[0]) - (1 - 300 * 4e-5)) < 1e-5 and torch.equal(w, s.split(s.master)[0].bfloat16())
    assert (lost == 1).all() and (w < 1).all()


def test_inference_tensors_and_views_of_one_buffer():
    with torch.inference_mode():
        w = torch.ones(300, device="cuda")
        s = pp.adamw_state([w])
        pp.adamw_step([w], [w * 0.5], s)
    assert (w < 1).all()
    flat = torch.randn(1000, device="cuda")
    params = [flat[:301], flat[301:640].view(3, 113), flat[640:]]
    ref = [p.clone() for p in params]
    grads = [torch.randn_like(p) for p in params]
    a, b = pp.adamw_state(params), pp.adamw_state(ref)
    pp.adamw_step(params, grads, a)
    pp.adamw_step(ref, grads, b)
    assert all(torch.equal(x, y) for x, y in zip(params, ref))


def test_embedding_trained_as_it_is_used():
    """embed, its gradient and the step, over a table, against the formulas in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(13)
    table = (torch.randn(50, 24, device="cuda", generator=g)).requires_grad_()
    ids = torch.randint(0, 50, (40, 30), device="cuda", generator=g)
    out = torch.randn(40, 30, 24, device="cuda", generator=g)
    s = pp.adamw_state([table])
    for t in range(1, 6):
        table.grad = None
        (pp.embed(ids, table, scale=2.0, padding_id=3) * out).sum().backward()
        grad, size = np.zeros((50, 24)), np.zeros((50, 24))
        np.add.at(grad, ids.cpu().numpy().ravel(), 2.0 * wide(out).reshape(-1, 24))
        np.add.at(size, ids.cpu().numpy().ravel(), 2.0 * np.abs(wide(out)).reshape(-1, 24))
        grad[3] = size[3] = 0
        most = torch.bincount(ids.flatten()).max().item()  # terms of a sum: each addition rounds once
        assert (np.abs(wide(table.grad) - grad) <= (most + 2) * R.U * size).all()
        before = wide(table), wide(s.split(s.exp_avg)[0]), wide(s.split(s.exp_avg_sq)[0])
        pp.adamw_step([table], None, s, lr=1e-2, weight_decay=0.05)
        ref, err = R.step(before[0], wide(table.grad), before[1], before[2], t, 1e-2, B1, B2, EPS, 0.05)
        for got, x, e in zip((table, s.split(s.exp_avg)[0], s.split(s.exp_avg_sq)[0]), ref, err):
            near(got, x, e, torch.float32, t)
    assert (table[3] != 0).all()  # padding takes no gradient, but decays
