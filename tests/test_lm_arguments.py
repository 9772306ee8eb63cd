"""Refusals of the language-model operators, which need no GPU: the library's
own checks of its arguments, and the binding's."""
import ctypes

import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp
import lm_ref as R

BIG = (1 << 31) - 65536


def test_option_struct_size():
    assert ctypes.sizeof(pp.lm.LogitOpts) == 152


def test_vocab_grammar_arguments():
    L, d = pp.lib(), pp.desc_csv()

    def call(off=1, chars=1, size=4, n=2, desc=d, end=-1, vec=1, allowed=1, stride=4):
        return L.pp_vocab_grammar(off, chars, size, n, ctypes.byref(desc) if desc else None, end, vec, allowed,
                                  stride, None)

    for bad in (dict(off=None), dict(chars=None), dict(desc=None), dict(end=2), dict(end=-2), dict(vec=None),
                dict(allowed=None), dict(n=33, stride=1), dict(desc=pp.desc_csv_enc("utf-8"))):
        assert call(**bad) == pp.PP_EINVAL, bad
    broken = pp.desc_csv()
    broken.delta[0][0] = 9
    assert call(desc=broken) == pp.PP_EINVAL
    assert call(n=BIG, stride=1 << 30) == pp.PP_ETOOLARGE
    assert call(n=0, off=None, chars=None, size=0, vec=None, allowed=None, stride=0) == pp.PP_OK


def test_grammar_states_arguments():
    L = pp.lib()

    def call(vec=1, n=2, ns=5, tokens=1, kind=2, rows=2, cols=3, stride=3, out=1, ostride=4):
        return L.pp_grammar_states(vec, n, ns, tokens, kind, rows, cols, stride, None, None, 0, 0, out, ostride, None)

    for bad in (dict(vec=None), dict(ns=0), dict(ns=17), dict(tokens=None), dict(kind=4), dict(kind=-1),
                dict(out=None), dict(ostride=3)):
        assert call(**bad) == pp.PP_EINVAL, bad
    for big in (dict(rows=BIG), dict(cols=BIG, ostride=1 << 32), dict(n=BIG)):
        assert call(**big) == pp.PP_ETOOLARGE, big
    assert call(rows=0, out=None, tokens=None) == pp.PP_OK


def test_logits_arguments():
    L = pp.lib()

    def call(x=16, kind=0, rows=2, vocab=40, stride=40, out=32, ostride=40, **opts):
        o = pp.lm.LogitOpts(**opts)
        return L.pp_logits(x, kind, rows, vocab, stride, ctypes.byref(o), out, ostride, None)

    mask = dict(d_allowed=16, allowed_stride=2, d_state=1, n_states=5)
    for bad in (dict(x=None), dict(out=None), dict(kind=3), dict(ostride=39), dict(x=17), dict(out=17),
                dict(out=16, stride=48, ostride=40), dict(d_history=16, history_type=9, history_cols=1),
                dict(d_bias_offsets=16, n_bias=1), dict(d_bias_offsets=16, n_bias=1, d_bias_tokens=16),
                dict(mask, d_state=None), dict(mask, n_states=0), dict(mask, n_states=17),
                dict(mask, allowed_stride=1)):
        assert call(**bad) == pp.PP_EINVAL, bad
    for big in (dict(rows=BIG), dict(vocab=BIG, ostride=BIG, stride=BIG),
                dict(d_history=16, history_type=2, history_cols=BIG), dict(n_bias=BIG),
                dict(rows=1 << 30, vocab=1 << 20, stride=1 << 20, ostride=1 << 20)):
        assert call(**big) == pp.PP_ETOOLARGE, big
    assert call(rows=0) == pp.PP_OK and call(vocab=0, x=None, out=None) == pp.PP_OK


def test_embed_arguments():
    L = pp.lib()

    def call(ids=16, kind=2, n=3, table=16, tt=0, vocab=4, dim=8, ts=8, out=32, ot=0, os=8):
        return L.pp_embed(ids, kind, 1, n, table, tt, vocab, dim, ts, 1.0, -1, out, ot, os, None)

    for bad in (dict(ids=None), dict(ids=17), dict(kind=4), dict(table=None), dict(table=18), dict(tt=3),
                dict(out=None), dict(out=34), dict(ot=-1), dict(os=7)):
        assert call(**bad) == pp.PP_EINVAL, bad
    for big in (dict(n=BIG), dict(vocab=BIG), dict(dim=BIG, os=BIG)):
        assert call(**big) == pp.PP_ETOOLARGE, big
    assert call(n=0, ids=None, out=None) == pp.PP_OK and call(dim=0) == pp.PP_OK


def test_embed_grad_arguments():
    L = pp.lib()

    def call(ids=16, kind=2, n=3, grad=16, gt=0, vocab=4, dim=8, out=32, ot=0, os=8, acc=0):
        return L.pp_embed_grad(ids, kind, 1, n, grad, gt, 8, vocab, dim, 1.0, -1, acc, out, ot, os, None)

    for bad in (dict(ids=None), dict(ids=18), dict(kind=4), dict(grad=None), dict(grad=17), dict(gt=3),
                dict(out=None), dict(out=33), dict(ot=7), dict(os=7)):
        assert call(**bad) == pp.PP_EINVAL, bad
    for big in (dict(n=BIG), dict(vocab=BIG), dict(dim=1 << 28, os=1 << 28)):
        assert call(**big) == pp.PP_ETOOLARGE, big
    assert call(vocab=0, out=None) == pp.PP_OK and call(n=0, acc=1, ids=None, grad=None) == pp.PP_OK


def test_binding_refuses_before_the_library():
    d = pp.desc_csv()
    off, chars = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.uint8)
    for args in ((off.long(), chars), (off, chars.int()), (off[:0], chars), (off[::2], chars), (off, chars[::2])):
        with pytest.raises(ValueError):
            pp.vocab_grammar(*args, d)
    for end in (2, -1):
        with pytest.raises(ValueError):
            pp.vocab_grammar(off, chars, d, end_id=end)
    with pytest.raises(ValueError):  # there is no path without a GPU
        pp.vocab_grammar(off, chars, d)
    g = pp.Grammar(torch.zeros(9, dtype=torch.int64), torch.zeros(5, 4, dtype=torch.int32), 9, d)
    for bad in (dict(vectors=torch.zeros(8, dtype=torch.int64)), dict(vectors=torch.zeros(9)),
                dict(allowed=torch.zeros(4, 4, dtype=torch.int32)), dict(allowed=torch.zeros(5, 0, dtype=torch.int32))):
        a = dict(dict(vectors=g.vectors, allowed=g.allowed), **bad)
        with pytest.raises(ValueError):
            pp.Grammar(a["vectors"], a["allowed"], 9, d)
    tokens = torch.zeros(2, 3, dtype=torch.int32)
    u8 = torch.zeros(2, dtype=torch.uint8)
    for kw in (dict(tokens=tokens[0]), dict(tokens=tokens.float()), dict(start=u8[:1]), dict(start=u8.int()),
               dict(lengths=torch.zeros(2)), dict(lengths=torch.zeros(1, dtype=torch.int32)),
               dict(out=torch.zeros(2, 3, dtype=torch.uint8)), dict(tokens=tokens.t())):
        with pytest.raises(ValueError):
            pp.grammar_states(g, **dict(dict(tokens=tokens), **kw))
    x = torch.zeros(2, 9)
    f2, i2 = torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(logits=x.double()), dict(logits=x[0]), dict(out=torch.zeros(2, 8)), dict(out=x.half()),
               dict(repetition=f2), dict(history=tokens[:1]), dict(history=tokens, history_len=f2),
               dict(history=tokens, repetition=i2), dict(history=tokens, repetition=f2[:1]),
               dict(history=tokens.float()), dict(grammar=g), dict(states=u8), dict(grammar=g, states=u8[:1]),
               dict(grammar=g, states=u8, logits=torch.zeros(2, 8)), dict(bias=(i2, i2, f2)),
               dict(bias=(torch.zeros(3, dtype=torch.int32), i2, f2[:1])), dict(logits=x.t())):
        with pytest.raises(ValueError):
            pp.process_logits(**dict(dict(logits=x), **kw))
    table, ids = torch.zeros(9, 8), torch.zeros(4, dtype=torch.int64)
    for kw in (dict(ids=ids.float()), dict(ids=ids.short()), dict(table=table[0]), dict(table=table.double()),
               dict(table=table.t()), dict(out=torch.zeros(4, 7)), dict(dtype=torch.float64),
               dict(out=torch.zeros(4, 8), dtype=torch.float16),
               dict(ids=torch.zeros(4, 6, dtype=torch.int64)[:, :3]),
               dict(table=table.clone().requires_grad_(), out=torch.zeros(4, 8))):
        with pytest.raises(ValueError):
            pp.embed(**dict(dict(ids=ids, table=table), **kw))
    grad = torch.zeros(4, 8)
    for kw in (dict(grad=grad[:3]), dict(grad=grad.double()), dict(grad=grad[:, 0]), dict(accumulate=True),
               dict(out=torch.zeros(9, 7)), dict(dtype=torch.int32), dict(grad=torch.zeros(8, 4).t())):
        with pytest.raises(ValueError):
            pp.embed_grad(**dict(dict(ids=ids, grad=grad, n_vocab=9), **kw))


def test_plain_forms_by_hand():
    """The tests' own 64-bit forms on cases worked out by hand."""
    to, fine = R.vocab([b"a", b'"', b"", b",", b'"x"', b"end"], pp.desc_csv(), end=5)
    assert to[0].tolist() == [1, 1, 2, 4, 4] and to[1].tolist() == [2, 4, 3, 2, 4]
    assert to[2].tolist() == [0, 1, 2, 3, 4] and to[4].tolist() == [3, 4, 4, 3, 4]
    assert fine[:, 5].tolist() == [True, True, False, True, False]
    assert fine[0].tolist() == [True, True, False, True, True, True] and not fine[4].any()
    st = R.states(to, np.array([[1, 0, 1, 9]]), 5, [0], [4])
    assert st.tolist() == [[0, 2, 2, 3, 255]]
    x, _ = R.logits(np.array([[2.0, -2.0, 1.0]]), history=np.array([[0, 1, 1]]), prompt_len=[1], repetition=[2.0],
                    presence=[0.5], frequency=[0.25], bias=([0, 1], [2], [3.0]))
    assert x.tolist() == [[1.0, -5.0, 4.0]]
    g, _ = R.embed_grad(np.array([1, 0, 1]), np.array([[1.0], [2.0], [4.0]]), 3, 2.0, 0)
    assert g.tolist() == [[0.0], [10.0], [0.0]]
