"""Every array of the language-model entry points lies at its type's
alignment: the library refuses others, which a kernel would fault on."""
import ctypes

import pytest

import dfa_parsing_delimiter_gb300 as pp


@pytest.mark.parametrize("which,off", [("offsets", 2), ("vectors", 4), ("allowed", 2)])
def test_vocab_grammar(which, off):
    a = {"offsets": 64, "vectors": 64, "allowed": 64}
    a[which] += off
    d = pp.desc_csv()
    assert pp.lib().pp_vocab_grammar(a["offsets"], 65, 4, 2, ctypes.byref(d), -1, a["vectors"], a["allowed"], 4,
                                     None) == pp.PP_EINVAL


@pytest.mark.parametrize("which,kind,off", [("vectors", 0, 4), ("tokens", 2, 2), ("tokens", 3, 4), ("lengths", 0, 2)])
def test_grammar_states(which, kind, off):
    a = {"vectors": 64, "tokens": 64, "lengths": 64}
    a[which] += off
    assert pp.lib().pp_grammar_states(a["vectors"], 2, 5, a["tokens"], kind, 2, 3, 3, a["lengths"], 65, 1, 0, 65, 4,
                                      None) == pp.PP_EINVAL


@pytest.mark.parametrize("which,off", [
    ("d_history", 2), ("d_history_row", 2), ("d_history_len", 1), ("d_prompt_len", 2), ("d_repetition", 2),
    ("d_presence", 1), ("d_frequency", 2), ("d_bias_offsets", 2), ("d_bias_tokens", 1), ("d_bias_values", 2),
    ("d_allowed", 2)])
def test_logits(which, off):
    pointers = [name for name, kind in pp.lm.LogitOpts._fields_ if name.startswith("d_")]
    a = {name: 64 for name in pointers}
    a[which] += off
    o = pp.lm.LogitOpts(**a, history_rows=2, history_cols=3, history_stride=3, n_bias=1, allowed_stride=2, state_stride=1,
                        n_states=5, history_type=2)
    assert pp.lib().pp_logits(64, 0, 2, 40, 40, ctypes.byref(o), 1 << 12, 40, None) == pp.PP_EINVAL


def test_logits_history_of_int64():
    o = pp.lm.LogitOpts(d_history=68, history_rows=2, history_cols=3, history_stride=3, d_presence=64, history_type=3)
    assert pp.lib().pp_logits(64, 0, 2, 40, 40, ctypes.byref(o), 1 << 12, 40, None) == pp.PP_EINVAL
