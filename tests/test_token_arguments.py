"""Refusals of the probabilities of tokens and of the verification of drafts,
which need no GPU, and the tests' own plain forms on cases worked out by hand."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp
import tokens_ref as R

BIG = (1 << 31) - 65536


def test_option_struct_size():
    assert ctypes.sizeof(pp.lm.DraftOpts) == 48


def test_token_probs_arguments():
    L = pp.lib()

    def call(x=16, kind=0, rows=2, vocab=40, stride=40, t=None, k=None, out=1 << 12, ostride=40):
        return L.pp_token_probs(x, kind, rows, vocab, stride, t, k, out, ostride, None)

    for bad in (dict(x=None), dict(out=None), dict(kind=3), dict(kind=-1), dict(ostride=39), dict(x=18), dict(out=(1 << 12) + 2),
                dict(t=2), dict(k=2), dict(x=1 << 12, stride=48), dict(x=1 << 12, kind=1), dict(x=1 << 12, kind=2, rows=1),
                dict(x=17, kind=1)):
        assert call(**bad) == pp.PP_EINVAL, bad
    for big in (dict(rows=BIG), dict(rows=BIG // 8), dict(vocab=1 << 30, stride=1 << 30, ostride=1 << 30)):
        assert call(**big) == pp.PP_ETOOLARGE, big
    assert call(rows=0, x=None, out=None) == pp.PP_OK and call(vocab=0, x=None, out=None) == pp.PP_OK


def test_verify_drafts_arguments():
    L = pp.lib()

    def call(target=16, kind=0, rows=20, vocab=40, stride=40, drafts=16, itype=2, n=2, k=3, ds=3, accept=16, accs=3,
             sample=16, tokens=16, ts=4, counts=16, **o):
        opts = pp.lm.DraftOpts(**o)
        return L.pp_verify_drafts(target, kind, rows, vocab, stride, drafts, itype, n, k, ds, accept, accs, sample,
                                  ctypes.byref(opts), tokens, ts, counts, None)

    for bad in (dict(target=None), dict(kind=3), dict(kind=-1), dict(itype=4), dict(itype=-1), dict(drafts=None),
                dict(accept=None), dict(sample=None), dict(tokens=None), dict(counts=None), dict(ts=3), dict(vocab=0),
                dict(target=18), dict(target=17, kind=1), dict(drafts=18), dict(drafts=20, itype=3), dict(accept=18),
                dict(sample=18), dict(tokens=18), dict(counts=18), dict(d_probs=18), dict(d_probs_row=18),
                dict(d_target_row=18), dict(d_lengths=18)):
        assert call(**bad) == pp.PP_EINVAL, bad
    for big in (dict(rows=BIG), dict(n=BIG // 8), dict(vocab=1 << 30), dict(k=1 << 24, ts=1 << 25),
                dict(d_probs=16, probs_rows=BIG)):
        assert call(**big) == pp.PP_ETOOLARGE, big
    assert call(n=0, target=None, drafts=None, tokens=None) == pp.PP_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="tensors of the CPU, which no kernel may get")
def test_binding_refuses_before_the_library(monkeypatch):
    x, f2, i2 = torch.zeros(2, 9), torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    target, q = torch.zeros(8, 9), torch.zeros(6, 9)
    drafts, accept, sample = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2)
    tokens, counts = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    good = dict(target=target, drafts=drafts, accept=accept, sample=sample)
    with pytest.raises(ValueError):  # there is no path without a GPU
        pp.token_probs(x)
    with pytest.raises(ValueError):
        pp.verify_drafts(**good)
    # past the check that there is one: what pp_bind refuses
    monkeypatch.setattr(pp.lm, "_call", lambda fn, what, like, stream, *args: fn(*args, 0))
    for kw in (dict(logits=x.double()), dict(logits=x[0]), dict(logits=x[None]), dict(out=torch.zeros(2, 8)), dict(out=x.half()),
               dict(out=torch.zeros(9, 2).t()), dict(temperature=f2[:1]), dict(temperature=i2), dict(temperature=x[:, 0]),
               dict(top_k=f2), dict(top_k=i2[:1]), dict(top_k=i2.long()), dict(logits=torch.zeros(9, 2).t()),
               dict(logits=x.clone().requires_grad_(), out=torch.zeros(2, 9)), dict(out=torch.zeros(2, 9, requires_grad=True))):
        with pytest.raises(ValueError):
            pp.token_probs(**dict(dict(logits=x), **kw))
    for kw in (dict(target=target.double()), dict(target=target[0]), dict(target=target[:7]), dict(target=torch.zeros(8, 0)),
               dict(target=torch.zeros(9, 8).t()), dict(drafts=drafts.float()), dict(drafts=drafts.short()), dict(drafts=drafts[0]),
               dict(drafts=torch.zeros(3, 2, dtype=torch.int32).t()), dict(accept=accept[:, :2]), dict(accept=accept.double()),
               dict(accept=torch.zeros(3, 2).t()), dict(sample=sample[:1]), dict(sample=sample.double()), dict(sample=None),
               dict(draft_probs=q[:5]), dict(draft_probs=q.half()), dict(draft_probs=q[:, :8]), dict(draft_probs=torch.zeros(9, 6).t()),
               dict(draft_probs=q, draft_row=i2[:1]), dict(draft_probs=q, draft_row=f2), dict(lengths=f2), dict(lengths=i2[:1]),
               dict(target_row=i2.long()), dict(target_row=i2[:1]), dict(out=(tokens[:, :3], counts)), dict(out=(tokens, counts[:1])),
               dict(out=(tokens.long(), counts)), dict(out=(tokens, counts.long())), dict(out=(tokens, counts[0])),
               dict(out=(tokens, torch.zeros(4, dtype=torch.int32)[::2])), dict(out=(torch.zeros(4, 2, dtype=torch.int32).t(), counts))):
        with pytest.raises(ValueError):
            pp.verify_drafts(**dict(good, **kw))


def test_cluster_blocks_have_started_before_remote_accesses():
    """As for the other kernels of clusters: what orders the first access to another block's
    shared memory after that block's start shows in the source alone."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dfa_parsing_delimiter_gb300", "csrc")
    with open(os.path.join(csrc, "pp_verify.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = [d for d in re.split(r"(?m)^\}", text) if "st.shared::cluster" in d]
    assert found
    for body in found:
        store = body.index("st.shared::cluster")
        assert 0 <= body.find("cluster_arrive(") < body.find("cluster_wait(") < store


def test_probabilities_by_hand():
    inf, nan = np.inf, np.nan
    x = np.array([[0.0, np.log(3.0), -inf, nan], [-inf, -inf, nan, -inf], [inf, 1.0, inf, 2.0], [2.0, 5.0, 5.0, 1.0],
                  [1.0, 1.0, 1.0, 1.0]])
    p, _ = R.probs(x, temperature=[1.0, 1.0, 1.0, 0.0, 2.0], top_k=[0, 1, 0, 0, 3])
    assert np.allclose(p, [[0.25, 0.75, 0, 0], [0, 0, 0, 0], [0.5, 0, 0.5, 0], [0, 1, 0, 0], [1 / 3, 1 / 3, 1 / 3, 0]])
    p, _ = R.probs(np.array([[0.0, np.log(4.0)]]), temperature=[2.0])
    assert np.allclose(p, [[1 / 3, 2 / 3]])


def test_verification_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0.0, 1.0, 0.0]])
    q = np.array([[0.25, 0.75, 0.0]])
    one = np.array([[1]])

    def go(u, s, **kw):
        a = dict(dict(target=p, drafts=one, accept=np.array([[u]]), sample=np.array([s]), draft_probs=q), **kw)
        t, c = R.verify(**a)
        return t[0].tolist(), int(c[0])

    assert go(0.3, 0.9) == ([1, 1], 2)  # 0.3 * 0.75 < 0.25; then the second row
    assert go(0.4, 0.4) == ([0, -1], 1)  # not: what is left is 0.25 of token 0 and 0.25 of token 2
    assert go(0.4, 0.5) == ([2, -1], 1)
    assert go(0.2, 0.1, draft_probs=None) == ([1, 1], 2) and go(0.25, 0.1, draft_probs=None) == ([0, -1], 1)
    assert go(0.9, 0.7, draft_probs=None) == ([2, -1], 1)  # the sure draft itself is left out
    assert go(0.9, 0.7, target=np.array([[0, 1e-20, 0.0], [0, 0, 1.0]])) == ([-1, -1], 0)  # less than a unit
    assert go(0.5, 0.3, lengths=[0]) == ([0, -1], 1) and go(0.5, 0.8, lengths=[0]) == ([2, -1], 1)
    assert go(0.5, 0.3, drafts=np.array([[7]])) == ([0, -1], 1)
    assert go(0.9, 0.5, target=np.array([[0.25, 0.75, 0], [0, 0, 1]]), draft_probs=np.array([[0.25, 1.0, 0]])) == ([1, -1], 1)
