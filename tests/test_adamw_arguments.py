"""Refusals of the AdamW step, which need no GPU, the layout of its state, and
the tests' own plain forms."""
import ctypes

import numpy as np
import pytest
import torch

import adamw_ref as R
import dfa_parsing_delimiter_gb300 as pp
from dfa_parsing_delimiter_gb300 import adamw as A


def test_struct_sizes():
    assert ctypes.sizeof(A.AdamWTensor) == 48 and ctypes.sizeof(A.AdamWStateStruct) == 72
    assert ctypes.sizeof(A.AdamWOpts) == 56


def test_adamw_arguments():
    L = pp.lib()

    def call(n_tensors=1, tensors=True, state=True, opts=True, t=None, s=None, o=None):
        a = dict(dict(d_param=16, d_grad=16, n=10, first=0, weight_decay=0.0, param_type=0, grad_type=0), **(t or {}))
        b = dict(dict(d_exp_avg=16, d_exp_avg_sq=16, d_exp_avg_exponent=1, d_exp_avg_sq_exponent=1, d_counters=4, n=512, bits=32),
                 **(s or {}))
        c = dict(dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8), **(o or {}))
        x, y, z = A.AdamWTensor(**a), A.AdamWStateStruct(**b), A.AdamWOpts(**c)
        return L.pp_adamw(ctypes.byref(x) if tensors else None, n_tensors, ctypes.byref(y) if state else None,
                          ctypes.byref(z) if opts else None, None)

    for bad in (dict(tensors=False), dict(state=False), dict(opts=False)):
        assert call(**bad) == pp.PP_EINVAL, bad
    for bad in (dict(d_param=None), dict(d_grad=None), dict(d_param=18), dict(d_grad=18), dict(param_type=1, d_param=17),
                dict(grad_type=2, d_grad=17), dict(param_type=3), dict(grad_type=-1), dict(first=100), dict(first=768),
                dict(n=513), dict(first=256, n=257), dict(n=2 ** 64 - 1), dict(first=2 ** 64 - 256),
                dict(weight_decay=float("nan")), dict(weight_decay=float("inf"))):
        assert call(t=bad) == pp.PP_EINVAL, bad
    for bad in (dict(bits=16), dict(bits=0), dict(n=500), dict(d_exp_avg=None), dict(d_exp_avg_sq=None), dict(d_exp_avg=24),
                dict(d_exp_avg_sq=20), dict(d_counters=None), dict(d_counters=6), dict(d_master=8),
                dict(bits=8, d_exp_avg_exponent=None), dict(bits=8, d_exp_avg_sq_exponent=None)):
        assert call(s=bad) == pp.PP_EINVAL, bad
    for bad in (dict(lr=-1e-3), dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1),
                dict(beta1=float("nan")), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1e-8), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(d_lr=6), dict(d_grad_scale=6), dict(d_skip=6)):
        assert call(o=bad) == pp.PP_EINVAL, bad
    assert call(s=dict(n=1 << 39)) == pp.PP_ETOOLARGE


def test_adamw_values_arguments():
    L = pp.lib()

    def call(kind=0, m=16, v=32, **s):
        st = A.AdamWStateStruct(**dict(dict(d_exp_avg=16, d_exp_avg_sq=16, d_exp_avg_exponent=1, d_exp_avg_sq_exponent=1, n=512,
                                            bits=8), **s))
        return L.pp_adamw_values(ctypes.byref(st), kind, m, v, None)

    for bad in (dict(kind=3), dict(kind=-1), dict(m=8), dict(v=8), dict(bits=32), dict(n=100), dict(d_exp_avg=None),
                dict(d_exp_avg_exponent=None)):
        assert call(**bad) == pp.PP_EINVAL, bad
    assert call(n=1 << 39) == pp.PP_ETOOLARGE
    assert call(n=0) == pp.PP_OK and call(m=None, v=None) == pp.PP_OK
    assert L.pp_adamw_values(None, 0, 16, 16, None) == pp.PP_EINVAL


def test_state_refuses_and_lays_out():
    w, b = torch.randn(3, 100), torch.randn(7)
    for bad in ([], [w.double()], [w.t()], [w, w], [w, w[1]], [w[:, ::2]], [w.clone().requires_grad_() * 2]):
        with pytest.raises(ValueError):
            pp.adamw_state(bad)
    with pytest.raises(ValueError):
        pp.adamw_state([w], bits=16)
    empty = torch.zeros(0, 4)
    s = pp.adamw_state([w, empty, b, torch.zeros(())], bits=8, master=True, seed=-1)
    assert s.first == (0, 512, 512, 768) and s.n == 1024 and s.sizes == (300, 0, 7, 1) and s.seed == 0xFFFFFFFF
    assert s.exp_avg.dtype == torch.uint8 and s.exp_avg_exponent.shape == (4,) and s.step.dim() == 0
    parts = s.split(s.master)
    assert torch.equal(parts[0], w) and torch.equal(parts[2], b) and parts[3].shape == ()
    other = pp.adamw_state([w, empty, b, torch.zeros(())], bits=8, master=True)
    other.exp_avg.fill_(3)
    other.step.fill_(41)
    s.load(**other.state_dict())
    assert torch.equal(s.exp_avg, other.exp_avg) and s.step == 41 and s._counters.tolist() == [41, 0]
    for bad in (dict(exp_avg=s.exp_avg[:-1]), dict(exp_avg=s.exp_avg.float()), dict(nothing=s.step), dict(step=s.step.float())):
        with pytest.raises(ValueError):
            s.load(**bad)
    with pytest.raises(ValueError):
        pp.adamw_state([w]).load(master=s.master)
    t = pp.adamw_state([w])
    assert t.values()[0] is t.exp_avg and t.values(torch.float16)[1].dtype == torch.float16
    with pytest.raises(ValueError):
        t.values(torch.float64)


@pytest.mark.skipif(torch.cuda.is_available(), reason="tensors of the CPU, which no kernel may get")
def test_binding_refuses_before_the_library(monkeypatch):
    w, b = torch.randn(3, 100), torch.randn(7)
    s = pp.adamw_state([w, b])
    gw, gb = torch.ones_like(w), torch.ones_like(b)
    one = torch.ones(())
    # past the check that there is a GPU: what pp_bind refuses
    monkeypatch.setattr(A, "_call", lambda fn, what, like, stream, *args: fn(*args, 0))
    good = dict(params=[w, b], grads=[gw, gb], state=s)
    for bad in (dict(params=[w]), dict(grads=[gw]), dict(params=[w, b, b]), dict(params=[b, w]), dict(grads=[gw.double(), gb]),
                dict(params=[w, b.int()]), dict(grads=[torch.ones(100, 3).t(), gb]), dict(grads=[torch.ones(3, 200)[:, ::2], gb]),
                dict(grads=[gw[:2], gb]), dict(weight_decay=[0.1]), dict(lr=-1.0), dict(lr=float("nan")), dict(lr=one.double()),
                dict(lr=torch.ones(2)), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0), dict(grad_scale=torch.ones(2)),
                dict(grad_scale=one.int()), dict(skip=one.bool()), dict(params=[w.clone().requires_grad_() * 1, b])):
        with pytest.raises(ValueError):
            pp.adamw_step(**dict(good, **bad))
    twice = pp.adamw_state([w, torch.zeros(3, 100)])
    with pytest.raises(ValueError, match="twice"):
        pp.adamw_step([w, w], [gw, gw], twice)
    monkeypatch.undo()
    with pytest.raises(ValueError):  # there is no path without a GPU
        pp.adamw_step(**good)


def test_plain_forms_by_hand():
    (p, m, v), _ = R.step(np.array([1.0]), np.array([2.0]), np.array([0.0]), np.array([0.0]), 1, 0.1, 0.9, 0.99, 0.0, 0.5)
    assert np.allclose([p[0], m[0], v[0]], [0.95 - 0.1, 0.2, 0.04])
    x = np.zeros(300, np.float32)
    x[:5] = [1.0, 1.5, -1.875, 0.03, 2.0 ** -13]
    c, e = R.encode(x, None, True)
    # 1 is at exponent 14, three bits behind the point: 0.03 = 1.92 * 2^-6 is nearest to 1.875 * 2^-6
    assert c[:5].tolist() == [14 * 8, 14 * 8 + 4, 128 + 14 * 8 + 7, 8 * 8 + 7, 8] and c[5:].max() == 0 and e.tolist() == [127, 1]
    assert R.value(c, e, True)[:5].tolist() == [1.0, 1.5, -1.875, 1.875 * 2.0 ** -6, 2.0 ** -13]
    c, e = R.encode(np.array([1.0, 1e-30, 0.0], np.float32), None, False)
    assert c.tolist() == [240, 1, 0]  # above 0: not rounded to it
    c, e = R.encode(np.array([1.0 + 1 / 16, 0.0], np.float32), np.array([32767, 65535], np.uint32), False)
    assert c.tolist() == [240, 0] and R.encode(np.float32([1.0 + 1 / 16]), np.array([32768]), False)[0].tolist() == [241]
    c, e = R.encode(np.array([np.inf, 1.0], np.float32), None, False)
    assert c.tolist() == [0, 0] and e.tolist() == [255]
