"""Plain 64-bit forms of the language-model operators, for the tests."""
import numpy as np
import torch

F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24  # half a unit in the last place of 32 bits
# rounding to the type: 2^-p relative with p significant bits (24, 11, 8), and
# half the least subnormal number where values get that small
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.float16: (2.0 ** -11, 2.0 ** -25),
         torch.bfloat16: (2.0 ** -8, 2.0 ** -134)}


def round_bound(ref, error, dtype):
    """The most that a value within `error` of ref may be off once rounded."""
    rel, least = ROUND[dtype]
    return error + rel * (np.abs(ref) + error) + least


def table_of(desc):
    """[256, n_states] next states of a descriptor."""
    b2g = np.frombuffer(bytes(desc.byte_to_group), np.uint8).astype(int)
    delta = np.array([[desc.delta[g][s] for s in range(desc.n_states)] for g in range(desc.n_groups)])
    return delta[b2g]


def live_of(desc):
    """States from which an accepting one can be reached, not through the invalid state."""
    t = table_of(desc)
    ok = {s for s in range(desc.n_states) if desc.accept_mask >> s & 1 and s != desc.invalid_state}
    while True:
        more = {s for s in range(desc.n_states) if s != desc.invalid_state and s not in ok
                and any(int(t[b, s]) in ok for b in range(256))}
        if not more:
            return ok
        ok |= more


def vocab(tokens, desc, end=None):
    """(states reached [n, n_states], allowed [n_states, n]) of byte strings."""
    t, live = table_of(desc), live_of(desc)
    n, ns = len(tokens), desc.n_states
    to = np.zeros((n, ns), int)
    fine = np.zeros((ns, n), bool)
    for v, token in enumerate(tokens):
        for s in range(ns):
            q = s
            if v != end:
                for b in token:
                    q = int(t[b, q])
            to[v, s] = q
            if v == end:
                fine[s, v] = s in live and bool(desc.accept_mask >> s & 1)
            else:
                fine[s, v] = len(token) > 0 and s in live and q in live
    return to, fine


def states(to, tokens, n_states, start, lengths):
    """[rows, cols + 1]; to: [n_vocab, n_states]."""
    rows, cols = tokens.shape
    out = np.zeros((rows, cols + 1), np.uint8)
    for r in range(rows):
        q = int(start[r])
        q = q if q < n_states else 255
        out[r, 0] = q
        for t in range(cols):
            if t < lengths[r] and q != 255:
                v = int(tokens[r, t])
                q = int(to[v, q]) if 0 <= v < len(to) else 255
            out[r, t + 1] = q
    return out


def logits(x, history=None, history_len=None, prompt_len=None, history_row=None, repetition=None,
           presence=None, frequency=None, bias=None, fine=None):
    """(values, the most that 32-bit arithmetic may be off); x: [rows, vocab]
    float64, fine: [rows, vocab] truth values or None."""
    x = x.astype(np.float64).copy()
    rows, vocab = x.shape
    error = np.zeros_like(x)
    for r in range(rows):
        if history is not None:
            h = r if history_row is None else int(history_row[r])
            line = history[h] if 0 <= h < len(history) else history[0][:0]
            size = len(line) if history_len is None else min(max(int(history_len[r]), 0), len(line))
            given = 0 if prompt_len is None else max(int(prompt_len[r]), 0)
            seen, said = set(), {}
            for t in range(size):
                v = int(line[t])
                if 0 <= v < vocab:
                    seen.add(v)
                    if t >= given:
                        said[v] = said.get(v, 0) + 1
            one = np.float64(1)
            rep = one if repetition is None else np.float64(repetition[r])
            pres = 0.0 if presence is None else np.float64(presence[r])
            freq = 0.0 if frequency is None else np.float64(frequency[r])
            for v in seen:
                y = x[r, v] / rep if x[r, v] > 0 else x[r, v] * rep
                size_of = abs(y)
                if v in said:
                    y = y - freq * said[v] - pres
                    size_of += abs(freq * said[v]) + abs(pres)
                x[r, v] = y
                error[r, v] += 4 * U32 * size_of
        if bias is not None:
            at, tokens, values = bias
            last = {}
            for e in range(max(int(at[r]), 0), min(int(at[r + 1]), len(tokens))):
                last[int(tokens[e])] = float(values[e])
            for v, b in last.items():
                if 0 <= v < vocab:
                    x[r, v] += b
                    error[r, v] += 2 * U32 * (abs(b) + abs(x[r, v]) + error[r, v])
    if fine is not None:
        x[~fine] = -np.inf
        error[~fine] = 0
    return x, error


def embed(ids, table, scale, pad):
    vocab = len(table)
    out = np.zeros((ids.size, table.shape[1]))
    there = (ids >= 0) & (ids < vocab) & (ids != (-1 if pad is None else pad))
    out[there] = table[ids[there]].astype(np.float64) * np.float64(np.float32(scale))
    return out


def embed_grad(ids, grad, vocab, scale, pad, old=None):
    """(values, the most that 32-bit sums may be off in any order)."""
    scale = np.float64(np.float32(scale))
    out = np.zeros((vocab, grad.shape[1]))
    size, count = np.zeros_like(out), np.zeros(vocab)
    for i, v in enumerate(ids.tolist()):
        if 0 <= v < vocab and v != pad:
            out[v] += grad[i]
            size[v] += np.abs(grad[i])
            count[v] += 1
    out, size = out * scale, size * abs(scale)
    error = (count[:, None] + 2) * U32 * size
    if old is not None:
        out = out + old
        error = error + 2 * U32 * (np.abs(out) + np.abs(old)) * (count[:, None] > 0)
    return out, error


def check(got, ref, error, dtype):
    """Every value within its bound; infinities and NaN in the same places."""
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    rest = ~fine & ~np.isnan(ref)
    assert np.array_equal(got[rest], ref[rest])
    off = np.abs(got[fine] - ref[fine])
    assert np.all(off <= round_bound(ref[fine], error[fine], dtype)), float((off - round_bound(ref[fine], error[fine], dtype)).max())
