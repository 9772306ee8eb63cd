"""The operators at the two ends of a language model (pp.h, "language models").

  pp_vocab_grammar / vocab_grammar    a vocabulary under a DFA -> Grammar
  pp_grammar_states / grammar_states  the DFA's state along token sequences
  pp_logits / process_logits          penalties, biases and the grammar's mask
  pp_token_probs / token_probs        logits as probabilities: temperature, top-k
  pp_verify_drafts / verify_drafts    drafted tokens against them; the next token
  pp_embed / embed                    rows of a table by id
  pp_embed_grad / embed_grad          the gradient for the table (both differentiable)

Argument marshalling only, as in the rest of the binding: shapes and types
are checked here (or in pp_bind, whose calls also take less of the time than
ctypes'), everything is computed by libpp's kernels on the given
stream (default: the current one).  New outputs belong to that stream; the
caller orders the use of every tensor on other streams, as with any kernel
launch.  Result tensors that are given count as written to in place: they may
not require a gradient while gradients are recorded.  Arguments that do not fit
raise ValueError, errors of the library RuntimeError.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from contextlib import nullcontext

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

import dfa_parsing_delimiter_gb300 as pp

FTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
ITYPE = {torch.uint8: 0, torch.int8: 1, torch.int32: 2, torch.int64: 3}
STATE_NONE = 0xFF
_U8 = (torch.uint8,)

_vp, _sz, _int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_i64, _f32 = ctypes.c_int64, ctypes.c_float


class LogitOpts(ctypes.Structure):
    """pp_logit_opts."""
    _fields_ = [("d_history", _vp), ("d_history_row", _vp), ("d_history_len", _vp),
                ("d_prompt_len", _vp), ("history_rows", _sz), ("history_cols", _sz),
                ("history_stride", _sz), ("d_repetition", _vp), ("d_presence", _vp),
                ("d_frequency", _vp), ("d_bias_offsets", _vp), ("d_bias_tokens", _vp),
                ("d_bias_values", _vp), ("n_bias", _sz), ("d_allowed", _vp),
                ("allowed_stride", _sz), ("d_state", _vp), ("state_stride", _sz),
                ("n_states", ctypes.c_int32), ("history_type", ctypes.c_int32)]


class DraftOpts(ctypes.Structure):
    """pp_draft_opts."""
    _fields_ = [("d_probs", _vp), ("d_probs_row", _vp), ("probs_rows", _sz), ("probs_stride", _sz),
                ("d_target_row", _vp), ("d_lengths", _vp)]


_NO_HISTORY, _NO_BIAS, _NO_GRAMMAR = (0,) * 10, (0,) * 4, (0,) * 5


def declare(L: ctypes.CDLL) -> None:
    """The entry points' argument types."""
    sigs = {
        "pp_vocab_grammar": [_vp, _vp, _sz, _sz, ctypes.POINTER(pp.DfaDesc), _i64, _vp, _vp, _sz, _vp],
        "pp_grammar_states": [_vp, _sz, _int, _vp, _int, _sz, _sz, _sz, _vp, _vp, _sz,
                              ctypes.c_uint8, _vp, _sz, _vp],
        "pp_logits": [_vp, _int, _sz, _sz, _sz, _vp, _vp, _sz, _vp],
        "pp_embed": [_vp, _int, _sz, _sz, _vp, _int, _sz, _sz, _sz, _f32, _i64, _vp, _int, _sz, _vp],
        "pp_embed_grad": [_vp, _int, _sz, _sz, _vp, _int, _sz, _sz, _sz, _f32, _i64, _int, _vp,
                          _int, _sz, _vp],
        "pp_embed_grad_noalloc": [_vp, _int, _sz, _sz, _vp, _int, _sz, _sz, _sz, _f32, _i64, _int, _vp,
                                  _int, _sz, _vp, _sz, _vp],
        "pp_embed_grad_scratch": [_sz, _sz, _sz],
        "pp_token_probs": [_vp, _int, _sz, _sz, _sz, _vp, _vp, _vp, _sz, _vp],
        "pp_verify_drafts": [_vp, _int, _sz, _sz, _sz, _vp, _int, _sz, _sz, _sz, _vp, _sz, _vp,
                             _vp, _vp, _sz, _vp, _vp],
    }
    for name, args in sigs.items():
        getattr(L, name).restype = _sz if name == "pp_embed_grad_scratch" else _int
        getattr(L, name).argtypes = args


_c = None  # pp_bind, from the first call on: checks and calls without ctypes' share of the time


def _lib():
    return _c if _c is not None else _load()


def _load():
    global _c
    from .build import BIND
    L = pp.lib()
    if not os.path.exists(BIND):
        raise RuntimeError(f"{BIND} not built; run __graft_entry__.build() (it needs Python's headers)")
    spec = importlib.util.spec_from_file_location(__package__ + ".pp_bind", BIND)
    bind = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bind)
    bind.init(*[ctypes.cast(getattr(L, "pp_" + name), _vp).value
                for name in ("vocab_grammar", "grammar_states", "logits", "embed", "embed_grad_noalloc", "embed_grad_scratch",
                              "token_probs", "verify_drafts", "adamw")])
    bind.types(*FTYPE, *ITYPE)  # in the order of their numbers
    _c = bind
    return bind


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _wrong(t, like, name: str, dtypes, ndim) -> None:
    raise ValueError(f"{name}: want {ndim} dimensions of {[str(d) for d in dtypes]} on {like.device}, "
                     f"got {tuple(t.shape)} of {t.dtype} on {t.device}")


def _on(t: torch.Tensor, like: torch.Tensor, name: str, dtypes, ndim: int) -> None:
    if t.dtype not in dtypes or t.dim() != ndim or t.get_device() != like.get_device():
        _wrong(t, like, name, dtypes, ndim)


def _on_stream(stream):
    """A context in which torch's own work goes to the call's stream."""
    return nullcontext() if stream is None else torch.cuda.stream(stream)


def _new(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _matrix_stride(t: torch.Tensor, name: str) -> int:
    """Row stride of a matrix with contiguous rows."""
    stride = t.stride()
    if stride[1] != 1 and t.size(1) > 1 and t.numel():
        raise ValueError(f"{name}: the last dimension has to be contiguous")
    return stride[0]


def _written(out: torch.Tensor) -> None:
    """Called where a kernel is about to write to a tensor of the caller's:
    autograd refuses a backward pass that needs what was there."""
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError("out: not one that requires a gradient")
    if not out.is_inference():
        increment_version(out)


def _call(fn, what: str, like: torch.Tensor, stream, *args) -> None:
    """One library call on the tensors' device and the stream."""
    dev = like.get_device()
    if dev < 0:
        raise ValueError(f"{what}: want tensors on a GPU, got {like.device}")
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        pp._check(rc, what)


def _followed(t: torch.Tensor) -> bool:
    """Whether autograd follows t, backward or forward."""
    return (t.requires_grad and torch.is_grad_enabled()) or \
        (forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None)


# ------------------------------------------------------------------ grammars
class Grammar:
    """A vocabulary under a DFA: `vectors` (int64 [n_vocab], a nibble per
    state), `allowed` (int32 [n_states, words], a bit per token), and the
    DFA's `start_state` and `accept_mask`.  vocab_grammar makes one."""

    def __init__(self, vectors: torch.Tensor, allowed: torch.Tensor, n_vocab: int, desc):
        _on(vectors, allowed, "vectors", (torch.int64,), 1)
        _on(allowed, allowed, "allowed", (torch.int32,), 2)
        self._set(vectors, allowed, int(n_vocab), desc)
        _need(vectors.is_contiguous() and vectors.size(0) == self.n_vocab, "vectors: want one a token")
        _need(allowed.size(0) == self.n_states and allowed.size(1) * 32 >= self.n_vocab
              and _matrix_stride(allowed, "allowed") >= allowed.size(1), "allowed: want a row a state")

    def _set(self, vectors, allowed, n_vocab, desc) -> None:
        self.vectors, self.allowed, self.n_vocab = vectors, allowed, n_vocab
        self.n_states, self.start_state, self.accept_mask = desc.n_states, desc.start_state, desc.accept_mask

    @classmethod
    def _of(cls, vectors, allowed, n_vocab, desc) -> "Grammar":
        g = cls.__new__(cls)
        g._set(vectors, allowed, n_vocab, desc)
        return g

    def accepts(self, states: torch.Tensor) -> torch.Tensor:
        """Whether texts that end in these states are complete."""
        s = states.to(torch.int64)
        return (s < self.n_states) & ((self.accept_mask >> s.clamp(max=31)) & 1).bool()


def vocab_grammar(offsets: torch.Tensor, chars: torch.Tensor, desc=None, end_id=None, stream=None) -> Grammar:
    """pp_vocab_grammar of a string column (int32 offsets and uint8 chars, as
    pp_parse writes one: token v is chars[offsets[v]:offsets[v + 1]]).
    end_id: the token that ends a text (None: there is none)."""
    desc = desc if desc is not None else pp.desc_csv()
    _on(offsets, chars, "offsets", (torch.int32,), 1)
    _on(chars, offsets, "chars", _U8, 1)
    _need(offsets.size(0) >= 1 and offsets.is_contiguous() and chars.is_contiguous(),
          "want contiguous offsets (one more than tokens) and chars")
    n = offsets.size(0) - 1
    _need(end_id is None or 0 <= end_id < n, f"end_id: want a token of the {n}, got {end_id}")
    words = -(-n // 128) * 4
    vectors = _new((n,), torch.int64, offsets, stream)
    allowed = _new((int(desc.n_states), words), torch.int32, offsets, stream)
    _call(_lib().vocab_grammar, "pp_vocab_grammar", offsets, stream, offsets.data_ptr(),
          chars.data_ptr(), chars.size(0), n, ctypes.addressof(desc), -1 if end_id is None else int(end_id),
          vectors.data_ptr(), allowed.data_ptr(), words)
    return Grammar._of(vectors, allowed, n, desc)


def grammar_states(grammar: Grammar, tokens: torch.Tensor, start=None, lengths=None, out=None,
                   stream=None) -> torch.Tensor:
    """pp_grammar_states: uint8 [rows, cols + 1], the state before each token
    of [rows, cols] token ids and after the last one.  start: uint8 [rows]
    (for instance an earlier result's last column) or None for the DFA's
    start state; lengths: int32 [rows], the tokens of each row that count."""
    _on(tokens, grammar.vectors, "tokens", ITYPE, 2)
    rows, cols = tokens.shape
    given = out
    if out is None:
        out = _new((rows, cols + 1), torch.uint8, tokens, stream)
    else:
        _on(out, tokens, "out", _U8, 2)
        _need(out.shape == (rows, cols + 1), "out: want one column more than tokens")
    ps, ss = 0, 0
    if start is not None:
        _on(start, tokens, "start", _U8, 1)
        _need(start.size(0) == rows, "start: want one state a row")
        ps, ss = start.data_ptr(), start.stride(0)
    if not rows:
        return out
    c = _lib()
    stride, ostride = _matrix_stride(tokens, "tokens"), _matrix_stride(out, "out")
    size = c.vec(lengths, torch.int32, tokens.get_device(), rows, "lengths")
    if given is not None:
        _written(out)
    _call(c.grammar_states, "pp_grammar_states", tokens, stream, grammar.vectors.data_ptr(), grammar.n_vocab,
          grammar.n_states, tokens.data_ptr(), ITYPE[tokens.dtype], rows, cols, stride, size, ps, ss,
          grammar.start_state, out.data_ptr(), ostride)
    return out


# ------------------------------------------------------------------ logits
class _Underived(torch.autograd.Function):
    @staticmethod
    def forward(ctx, call, arguments, *followed):
        ctx.what = call.__name__
        return call(*arguments)  # autograd follows nothing in here

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.what} has no derivative: detach its arguments")

    jvp = backward


def process_logits(logits: torch.Tensor, history=None, history_len=None, prompt_len=None, history_row=None,
                   repetition=None, presence=None, frequency=None, bias=None, grammar=None, states=None,
                   out=None, stream=None) -> torch.Tensor:
    """pp_logits of [rows, n_vocab] logits; `out` may be `logits` itself.
    history: [sequences, cols] token ids, of which row r counts the first
    history_len[r] of sequence history_row[r] (default: r), the first
    prompt_len[r] of them as given and the rest as answered.  repetition,
    presence, frequency: float32 [rows].  bias: (offsets int32 [rows + 1],
    tokens int32, values float32), an entry list per row.  grammar and states
    (uint8 [rows]): tokens that the state does not allow become -inf.  There
    is no derivative: a result of values that require a gradient raises
    RuntimeError when it is differentiated (and such values take no `out`)."""
    if forward_ad._current_level >= 0 or logits.requires_grad or (bias is not None and bias[-1].requires_grad) or (
            repetition is not None and repetition.requires_grad) or (presence is not None and presence.requires_grad) or (
            frequency is not None and frequency.requires_grad):
        values = (logits, repetition, presence, frequency, None if bias is None else bias[-1])
        followed = [t for t in values if t is not None and _followed(t)]
        if followed:
            _need(out is None, "out: not for values that require a gradient")
            return _Underived.apply(process_logits, (logits, history, history_len, prompt_len, history_row, repetition, presence,
                                                     frequency, bias, grammar, states, None, stream), *followed)
    _need(logits.dtype in FTYPE and logits.dim() == 2, "logits: want 2 dimensions of float32, float16 or bfloat16")
    rows, vocab = logits.shape
    dev, i32, f32 = logits.get_device(), torch.int32, torch.float32
    c = _lib()
    vec = c.vec
    given = out
    if out is None:
        out = torch.empty_like(logits) if stream is None and logits.is_contiguous() else \
            _new((rows, vocab), logits.dtype, logits, stream)
    else:
        _on(out, logits, "out", (logits.dtype,), 2)
        _need(out.shape == logits.shape, "out: want the shape of the logits")
    hist, itype = _NO_HISTORY, 0
    if history is not None:
        _on(history, logits, "history", ITYPE, 2)
        itype = ITYPE[history.dtype]
        lines, cols = history.shape
        _need(history_row is not None or lines >= rows, "history: want a row for each row of logits")
        hist = (history.data_ptr(), vec(history_row, i32, dev, rows, "history_row"),
                vec(history_len, i32, dev, rows, "history_len"),
                vec(prompt_len, i32, dev, rows, "prompt_len"),
                lines, cols, _matrix_stride(history, "history"),
                vec(repetition, f32, dev, rows, "repetition"),
                vec(presence, f32, dev, rows, "presence"),
                vec(frequency, f32, dev, rows, "frequency"))
    elif repetition is not None or presence is not None or frequency is not None:
        raise ValueError("penalties need a history")
    lists = _NO_BIAS
    if bias is not None:
        at, tokens, values = bias
        n = tokens.numel()
        _need(values.numel() == n, "bias: want as many values as tokens")
        lists = (vec(at, i32, dev, rows + 1, "bias offsets"), vec(tokens, i32, dev, n, "bias tokens"),
                 vec(values, f32, dev, n, "bias values"), n)
    mask = _NO_GRAMMAR
    if grammar is not None and states is not None:
        _on(states, logits, "states", _U8, 1)
        allowed = grammar.allowed
        if states.numel() != rows or grammar.n_vocab != vocab or allowed.get_device() != dev:
            raise ValueError(f"want {rows} states, and a grammar of {vocab} tokens on the logits' device")
        mask = (allowed.data_ptr(), allowed.stride(0), states.data_ptr(), states.stride(0), grammar.n_states)
    elif grammar is not states:
        raise ValueError("a grammar needs states, and states a grammar")
    if rows and vocab:
        stride, ostride = _matrix_stride(logits, "logits"), _matrix_stride(out, "out")
        if given is not None:
            _written(out)
        _call(c.logits, "pp_logits", logits, stream, logits.data_ptr(), FTYPE[logits.dtype], rows, vocab,
              stride, *hist, *lists, *mask, itype, out.data_ptr(), ostride)
    return out


# ------------------------------------------------------------------ tokens
def token_probs(logits: torch.Tensor, temperature=None, top_k=None, out=None, stream=None) -> torch.Tensor:
    """pp_token_probs of [rows, n_vocab] logits: float32 probabilities.
    temperature: float32 [rows] (not above 0: all at the largest logit);
    top_k: int32 [rows], how many of the most likely tokens stay (below 1:
    all).  `out` may be float32 logits themselves.  There is no derivative: a
    result of values that require a gradient raises RuntimeError when it is
    differentiated (and such values take no `out`)."""
    if forward_ad._current_level >= 0 or logits.requires_grad or (temperature is not None and temperature.requires_grad):
        followed = [t for t in (logits, temperature) if t is not None and _followed(t)]
        if followed:
            _need(out is None, "out: not for values that require a gradient")
            return _Underived.apply(token_probs, (logits, temperature, top_k, None, stream), *followed)
    if out is None:
        out = _new(logits.shape, torch.float32, logits, stream)
    else:
        _written(out)
    _call(_lib().token_probs, "pp_token_probs", logits, stream, logits, temperature, top_k, out)
    return out


def verify_drafts(target: torch.Tensor, drafts: torch.Tensor, accept: torch.Tensor, sample: torch.Tensor,
                  draft_probs=None, lengths=None, target_row=None, draft_row=None, out=None,
                  stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """pp_verify_drafts: (tokens int32 [n, k + 1], counts int32 [n]), the
    accepted ones of [n, k] drafted tokens and the one that follows them, then
    -1; without drafts (k or a length of 0) one drawn token.  target: [rows,
    n_vocab] probabilities, of which request r has k + 1 rows from
    target_row[r] on (default: r * (k + 1)); draft_probs: the rows that its
    drafts were drawn from, k from draft_row[r] on (default: r * k), or None
    for drafts without a choice; lengths: int32 [n], the drafts of each request
    that count; accept: float32 [n, k] and sample: float32 [n], random numbers
    in [0, 1).  out: (tokens, counts) to write to."""
    n, k = drafts.shape
    if out is None:
        tokens, counts = _new((n, k + 1), torch.int32, target, stream), _new((n,), torch.int32, target, stream)
    else:
        tokens, counts = out
        _need(counts.shape == (n,), "out: want a count for each request")
        _written(tokens)
        _written(counts)
    _call(_lib().verify_drafts, "pp_verify_drafts", target, stream, target, drafts, accept, sample, draft_probs, lengths,
          target_row, draft_row, tokens, counts)
    return tokens, counts


# ------------------------------------------------------------------ embedding
def _flat_ids(ids: torch.Tensor) -> tuple[int, int]:
    """(number of ids, their stride) of ids that lie at one stride."""
    _need(ids.dtype in ITYPE, "ids: want uint8, int8, int32 or int64")
    n = ids.numel()
    if ids.is_contiguous():
        return n, 1
    stride, want = None, 0
    for size, step in zip(reversed(ids.shape), reversed(ids.stride())):
        if size == 1:
            continue
        if stride is None:
            stride, want = step, step
        _need(step == want, "ids: want one stride over all dimensions")
        want = step * size
    return n, 1 if stride is None else stride


def _embed(ids, table, scale, padding_id, out, dtype, stream) -> torch.Tensor:
    n, stride = _flat_ids(ids)
    _on(table, ids, "table", FTYPE, 2)
    vocab, dim = table.shape
    shape = (*ids.shape, dim)
    given = out
    if out is None:
        out = _new(shape, dtype if dtype is not None else table.dtype, ids, stream)
    else:
        _need(out.dtype in FTYPE and out.device == ids.device and out.shape == shape and
              out.is_contiguous() and dtype in (None, out.dtype), "out: want the ids' shape and the width, contiguous")
    _need(out.dtype in FTYPE, "dtype: want float32, float16 or bfloat16")
    if n and dim:
        tstride = _matrix_stride(table, "table")
        if given is not None:
            _written(out)
        _call(_lib().embed, "pp_embed", ids, stream, ids.data_ptr(), ITYPE[ids.dtype], stride, n,
              table.data_ptr(), FTYPE[table.dtype], vocab, dim, tstride, scale,
              -1 if padding_id is None else padding_id, out.data_ptr(), FTYPE[out.dtype], dim)
    return out


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t with contiguous rows, as derivatives do not always come."""
    return t if t.stride(-1) == 1 else t.contiguous()


class _Embed(torch.autograd.Function):
    """embed is linear in the table and embed_grad its derivative, and the
    other way round: so derivatives of every order are calls of the two."""

    @staticmethod
    def forward(ctx, table, ids, scale, padding_id, dtype, stream):
        ctx.save_for_backward(ids)
        ctx.save_for_forward(ids)
        ctx.rest = (table.size(0), scale, padding_id, table.dtype, dtype)
        return _embed(ids, table, scale, padding_id, None, dtype, stream)

    @staticmethod
    def backward(ctx, grad):
        vocab, scale, padding_id, dtype, _ = ctx.rest
        return embed_grad(ctx.saved_tensors[0], _rows(grad), vocab, scale, padding_id, dtype=dtype), *[None] * 5

    @staticmethod
    def jvp(ctx, table, *rest):
        return embed(ctx.saved_tensors[0], _rows(table), ctx.rest[1], ctx.rest[2], dtype=ctx.rest[4])


class _EmbedGrad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad, ids, n_vocab, scale, padding_id, dtype, stream):
        ctx.save_for_backward(ids)
        ctx.save_for_forward(ids)
        ctx.rest = (scale, padding_id, grad.dtype, n_vocab, dtype)
        return _embed_grad(ids, grad, n_vocab, scale, padding_id, None, False, dtype, stream)

    @staticmethod
    def backward(ctx, grad):
        scale, padding_id, dtype = ctx.rest[:3]
        return embed(ctx.saved_tensors[0], _rows(grad), scale, padding_id, dtype=dtype), *[None] * 6

    @staticmethod
    def jvp(ctx, grad, *rest):
        scale, padding_id, _, vocab, dtype = ctx.rest
        return embed_grad(ctx.saved_tensors[0], _rows(grad), vocab, scale, padding_id, dtype=dtype)


def embed(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, padding_id=None, out=None, dtype=None,
          stream=None) -> torch.Tensor:
    """pp_embed: scale * table[ids], [*ids.shape, dim] in `dtype` (default:
    the table's).  ids: integers of any shape at one stride; padding_id and
    ids outside the table give zeros.  A table that requires a gradient gets
    it through embed_grad, and one with a tangent passes it on (then without
    `out`)."""
    if _followed(table):
        _need(out is None, "out: not for a table that requires a gradient")
        return _Embed.apply(table, ids, scale, padding_id, dtype, stream)
    return _embed(ids, table, scale, padding_id, out, dtype, stream)


def _embed_grad(ids, grad, n_vocab, scale, padding_id, out, accumulate, dtype, stream) -> torch.Tensor:
    n, stride = _flat_ids(ids)
    _need(grad.dtype in FTYPE and grad.device == ids.device and grad.dim() == ids.dim() + 1
          and grad.shape[:-1] == ids.shape, "grad: want the ids' shape and a last dimension")
    dim = grad.size(-1)
    if grad.dim() != 2:
        with _on_stream(stream):  # where this copies, the copy is the stream's
            grad = grad.reshape(n, dim)
    given = out
    if out is None:
        _need(not accumulate, "accumulate: needs an out")
        out = _new((n_vocab, dim), dtype if dtype is not None else grad.dtype, ids, stream)
    else:
        _on(out, ids, "out", FTYPE, 2)
        _need(out.shape == (n_vocab, dim) and dtype in (None, out.dtype), "out: want a row a token, of the width")
    _need(out.dtype in FTYPE, "dtype: want float32, float16 or bfloat16")
    if n_vocab and dim:
        gstride, ostride = _matrix_stride(grad, "grad"), _matrix_stride(out, "out")
        c = _lib()
        size = c.embed_grad_scratch(n, n_vocab, dim)
        scratch = _new((size,), torch.uint8, ids, stream) if size else None
        if given is not None:
            _written(out)
        _call(c.embed_grad, "pp_embed_grad", ids, stream, ids.data_ptr(), ITYPE[ids.dtype],
              stride, n, grad.data_ptr(), FTYPE[grad.dtype], gstride, n_vocab, dim,
              scale, -1 if padding_id is None else padding_id, int(bool(accumulate)), out.data_ptr(),
              FTYPE[out.dtype], ostride, 0 if scratch is None else scratch.data_ptr(), size)
    return out


def embed_grad(ids: torch.Tensor, grad: torch.Tensor, n_vocab: int, scale: float = 1.0, padding_id=None,
               out=None, accumulate: bool = False, dtype=None, stream=None) -> torch.Tensor:
    """pp_embed_grad: [n_vocab, dim], the gradient of embed's table from that
    of its result ([*ids.shape, dim]), in `dtype` (default: the gradient's).
    With accumulate it is added to `out`; else `out` is overwritten.  A
    gradient that requires one itself gets it through embed (then without
    `out`)."""
    if _followed(grad):
        _need(out is None, "out: not for a gradient that requires a gradient")
        _need(not accumulate, "accumulate: needs an out")
        return _EmbedGrad.apply(grad, ids, n_vocab, scale, padding_id, dtype, stream)
    return _embed_grad(ids, grad, n_vocab, scale, padding_id, out, accumulate, dtype, stream)
