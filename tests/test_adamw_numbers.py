"""Rates, eps and decays that 32 bits do not hold are refused: as infinities they would
make the parameters NaN."""
import ctypes

import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp
from dfa_parsing_delimiter_gb300 import adamw as A

INF, NAN = float("inf"), float("nan")


def test_the_library_refuses():
    L = pp.lib()

    def call(**o):
        x = A.AdamWTensor(d_param=16, d_grad=16, n=10, first=0)
        s = A.AdamWStateStruct(d_exp_avg=16, d_exp_avg_sq=16, d_counters=4, n=512, bits=32)
        o = A.AdamWOpts(**dict(dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8), **o))
        return L.pp_adamw(ctypes.byref(x), 1, ctypes.byref(s), ctypes.byref(o), None)

    for bad in (dict(lr=1e39), dict(lr=1e300), dict(eps=1e39), dict(eps=1e300)):
        assert call(**bad) == pp.PP_EINVAL, bad


@pytest.mark.skipif(torch.cuda.is_available(), reason="tensors of the CPU, which no kernel may get")
def test_the_binding_refuses(monkeypatch):
    w = torch.randn(3, 100)
    s = pp.adamw_state([w, w.clone()])
    monkeypatch.setattr(A, "_call", lambda fn, what, like, stream, *args: fn(*args, 0))
    for bad in (dict(lr=1e39), dict(eps=1e39), dict(weight_decay=1e39), dict(weight_decay=INF), dict(weight_decay=NAN),
                dict(weight_decay=[0.1, -1e39])):
        with pytest.raises(ValueError):
            pp.adamw_step([w, w.clone()], [w, w], s, **bad)
