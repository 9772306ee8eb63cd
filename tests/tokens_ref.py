"""Plain 64-bit forms of the probabilities of tokens and of the verification of
drafts, for the tests."""
import numpy as np

U = 2.0 ** -24  # half a unit in the last place of 32 bits


def kept(x, k):
    """Which logits of a row stay: the k largest, of equal ones the lowest tokens."""
    there = x > -np.inf  # false for NaN
    if 0 < k < x.size:
        y = np.where(np.isnan(x), -np.inf, x)
        order = np.argsort(-y, kind="stable")
        first = np.zeros(x.size, bool)
        first[order[:k]] = True
        there &= first
    return there


def probs(x, temperature=None, top_k=None):
    """(probabilities, the most that 32-bit arithmetic may be off), of [rows,
    vocab] logits in float64.

    With u = 2^-24 and y = (x - max) / T: the difference, log2(e), its quotient
    with T and the product are four roundings of the exponent, so 4 |y| u of the
    exponential, and exp2f is within 2 ulp, 4 u.  A sum of positive terms is off
    by what its terms are, at most that twice over where a part's sum is brought
    to the row's maximum (whose distance is no more than |y|), and by u for each
    addition on a term's way: at most one for every 256 values and 64 beyond.
    The reciprocal and the product add 3 u at most."""
    out, err = np.zeros_like(x), np.zeros_like(x)
    for r in range(len(x)):
        t = 1.0 if temperature is None else float(temperature[r])
        there = kept(x[r], 0 if top_k is None else int(top_k[r]))
        if not there.any():
            continue
        top = x[r][there].max()
        if not t > 2.0 ** -125:
            out[r, int(np.argmax(np.where(np.isnan(x[r]), -np.inf, x[r])))] = 1.0
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            y = np.where(x[r] == top, 0.0, (x[r] - top) / t)
        e = np.where(there, np.exp(np.where(there, y, 0.0)), 0.0)
        z = e.sum()
        size = np.where(there, np.minimum(np.abs(np.where(there, y, 0.0)), 1e4), 0.0)
        term = (4 * size + 4) * U
        total = (e * 2 * term).sum() / z + (x.shape[1] / 256 + 64) * U
        out[r] = e / z
        err[r] = out[r] * (term + total + 3 * U) * 1.01 + np.where(there, 2.0 ** -140, 0.0)
    return out, err


def units(p, bits):
    """Probabilities as whole numbers of 2^-bits, rounded down."""
    p = np.clip(np.nan_to_num(p.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)
    return np.floor(p * 2.0 ** bits).astype(np.int64)  # a power of two: exact


def verify(target, drafts, accept, sample, draft_probs=None, lengths=None, target_row=None, draft_row=None):
    """(tokens, counts) by Python's whole numbers."""
    n, k = drafts.shape
    rows, vocab = target.shape
    bits = 62 - (vocab - 1).bit_length()
    tokens, counts = np.full((n, k + 1), -1, np.int64), np.zeros(n, np.int64)

    def cut(p):
        return min(max(float(p), 0.0), 1.0) if p == p else 0.0

    for r in range(n):
        size = k if lengths is None else min(max(int(lengths[r]), 0), k)
        first = r * (k + 1) if target_row is None else int(target_row[r])
        qfirst = r * k if draft_row is None else int(draft_row[r])

        def row(i):
            return target[i] if 0 <= i < rows else None

        def qrow(i):
            return draft_probs[i] if 0 <= i < len(draft_probs) else None

        j = 0
        while j < size:
            d, u, p = int(drafts[r, j]), float(accept[r, j]), row(first + j)
            q = None if draft_probs is None else qrow(qfirst + j)
            if not (0 <= d < vocab) or p is None or not u >= 0 or (draft_probs is not None and q is None):
                break
            if not u * (1.0 if q is None else cut(q[d])) < cut(p[d]):  # 24 by 24 bits: exact in 64
                break
            j += 1
        p = row(first + j)
        whole = np.zeros(vocab, np.int64) if p is None else units(p, bits)
        w = whole.copy()
        if j < size:
            if draft_probs is None:
                if 0 <= int(drafts[r, j]) < vocab:
                    w[int(drafts[r, j])] = 0
            else:
                q = qrow(qfirst + j)
                if q is not None:
                    w = np.maximum(whole - units(q, bits), 0)
            if not w.any():
                w = whole
        total = int(w.sum())
        tokens[r, :j] = drafts[r, :j]
        counts[r] = j
        if total:
            s = float(sample[r])
            s = 0 if not s > 0 else 2 ** 31 - 1 if s >= 1 else int(s * 2 ** 31)
            tokens[r, j] = int(np.searchsorted(np.cumsum(w), total * s >> 31, side="right"))
            counts[r] += 1
    return tokens, counts
