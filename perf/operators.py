"""Cases for the operators between a language model and the DFAs of this
framework: a vocabulary read by a DFA, the DFA's states along token
sequences, the logits under penalties, biases and that grammar, and the
embedding of parsed ids with its gradient.

Every operator has a plain form here (elementary torch operations in 32 bits,
rounded once at the end) and, with `own` set, the framework's call.
"""
import math

import numpy as np
import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

FLOAT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NONE_STATE = 255  # the state of a row after a token outside the vocabulary


def listed():
    return [
        # the words of a small table of names, under the quoted-CSV rules
        {"name": "vocab csv 4k", "op": "vocab", "dfa": "csv", "vocab": 4099, "mean": 4},
        # a large subword vocabulary under the 16-state lexer
        {"name": "vocab json 256k", "op": "vocab", "dfa": "json", "vocab": 262144, "mean": 8},
        # one decode step of a full batch: one token a row
        {"name": "states decode 512x1", "op": "states", "dfa": "json", "vocab": 131072, "rows": 512,
         "cols": 1, "ragged": False},
        # long documents checked in one call, rows of unlike lengths
        {"name": "states 16x65537", "op": "states", "dfa": "csv", "vocab": 50001, "rows": 16,
         "cols": 65537, "ragged": True},
        # one user, short history: the smallest call that answers with a token
        {"name": "logits 1x32000 f32", "op": "logits", "type": "f32", "dfa": "csv", "rows": 1,
         "vocab": 32000, "history": 37, "bias": 5},
        # a serving batch with ordinary histories
        {"name": "logits 64x131072 bf16", "op": "logits", "type": "bf16", "dfa": "json",
         "rows": 64, "vocab": 131072, "history": 2047, "bias": 20},
        # the largest batch, an odd vocabulary (rows start at odd places), long histories
        {"name": "logits 512x131075 f16", "op": "logits", "type": "f16", "dfa": "csv",
         "rows": 512, "vocab": 131075, "history": 8191, "bias": 300},
        # one decode step's tokens into vectors
        {"name": "embed 64x4096 bf16", "op": "embed", "type": "bf16", "out": "bf16", "n": 64,
         "vocab": 131072, "dim": 4096},
        # a training batch's tokens, 32-bit weights, 16-bit activations
        {"name": "embed 65536x4096 f32", "op": "embed", "type": "f32", "out": "bf16",
         "n": 65536, "vocab": 65536, "dim": 4096},
        # categories of a parsed table: few ids, odd width
        {"name": "grad 333x257 f32", "op": "grad", "type": "f32", "out": "f32", "n": 333,
         "vocab": 4099, "dim": 257},
        # one sequence batch of a small model
        {"name": "grad 8192x1024 bf16", "op": "grad", "type": "bf16", "out": "f32", "n": 8192,
         "vocab": 32000, "dim": 1024},
        # a training batch of a large model
        {"name": "grad 131072x2048 bf16", "op": "grad", "type": "bf16", "out": "f32",
         "n": 131072, "vocab": 131072, "dim": 2048},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["vocab", "states", "logits", "embed", "grad"])
    dfa = rng.choice(["csv", "json"])
    if op == "vocab":
        return {"op": op, "dfa": dfa, "vocab": log(256, 262144), "mean": rng.randint(2, 8)}
    if op == "states":
        cols = log(1, 65537)
        return {"op": op, "dfa": dfa, "vocab": log(300, 131072), "rows": log(1, max(1, min(512, 2 ** 20 // cols))),
                "cols": cols, "ragged": rng.random() < 0.5}
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "logits":
        vocab = log(300, 131075)
        most = 512 * 131075 * 2 // SIZE[kind] // vocab
        return {"op": op, "type": kind, "dfa": dfa, "rows": log(1, min(most, 512)), "vocab": vocab,
                "history": log(1, 8191), "bias": log(1, 300)}
    out = rng.choice(["f32", "f16", "bf16"])
    if op == "embed":
        dim = log(8, 4096)
        return {"op": op, "type": kind, "out": out, "n": log(1, 65536), "vocab": log(300, 65536), "dim": dim}
    dim = log(8, 2048)
    return {"op": op, "type": kind, "out": rng.choice(["f32", kind]), "n": log(1, 131072),
            "vocab": log(300, 131072), "dim": dim}


# ------------------------------------------------------------------ the DFAs
def csv_rows():
    """Next state by (byte, state) of quoted CSV: at a boundary, in a field,
    in quotes, after a quote in quotes, invalid; and the accepting states."""
    t = np.tile(np.arange(16), (256, 1))
    t[:, :5] = [1, 1, 2, 4, 4]
    for b in b",\n":
        t[b, :5] = [0, 0, 2, 0, 4]
    t[ord('"'), :5] = [2, 4, 3, 2, 4]
    return t, 5, 0, 4, [0, 1, 3]


def json_rows():
    """The same of a lexer for JSON-like text: 0 start, 1 white space, 2
    punctuation, 3 and 4 in a string, 5 after a backslash, 6 after a string,
    7 minus, 8 zero, 9 integer, 10 point, 11 fraction, 12 to 14 exponent,
    15 invalid."""
    t = np.full((256, 16), 15)
    first = {b: 1 for b in b" \t\n\r"}
    first.update({b: 2 for b in b"{}[],:"})
    first.update({ord('"'): 3, ord("-"): 7, ord("0"): 8})
    first.update({b: 9 for b in b"123456789"})
    for b, s in first.items():
        t[b, [0, 1, 2, 6]] = s
        if b not in b"0123456789":
            t[b, [8, 9, 11, 14]] = s
    t[:, [3, 4, 5]] = 4
    t[ord('"'), [3, 4]] = 6
    t[ord("\\"), [3, 4]] = 5
    for b in b"0123456789":
        t[b, 7] = 8 if b == 48 else 9
        t[b, [9, 10, 11, 12, 13, 14]] = [9, 11, 11, 14, 14, 14]
    t[ord("."), [8, 9]] = 10
    for b in b"eE":
        t[b, [8, 9, 11]] = 12
    for b in b"+-":
        t[b, 12] = 13
    return t, 16, 0, 15, [0, 1, 2, 6, 8, 9, 11, 14]


ROWS = {"csv": csv_rows, "json": json_rows}


def vocabulary(n, mean, rs):
    """Random token strings (offsets, bytes): single bytes first, then words,
    numbers, white space and structural pieces, a few very long; some empty
    ones stand for special tokens, the last of which ends a text."""
    sizes = 1 + rs.geometric(1.0 / max(1.0, mean - 1), n)
    sizes = np.minimum(sizes, 64)
    sizes[rs.randint(0, n, max(1, n // 2000))] = rs.randint(65, 257, max(1, n // 2000))
    sizes[:256] = 1
    sizes[rs.randint(0, n, 8)] = 0
    sizes[n - 1] = 0
    off = np.zeros(n + 1, np.int64)
    off[1:] = np.cumsum(sizes)
    total = int(off[-1])
    of = np.repeat(np.arange(n), sizes)
    kind = rs.choice(4, n, p=[0.62, 0.2, 0.06, 0.12])[of]
    pools = [b"etaoinshrdlucmfwypvbgkjqxzETAOINS \xc3\xa9\xe2\x80", b"0123456789.0123456789e-", b"   \n\t ",
             b'{}[],:"\\",\n etaoinshr0123456789']
    pools = [np.frombuffer(p, np.uint8) for p in pools]
    chars = np.zeros(total, np.uint8)
    for k, p in enumerate(pools):
        at = np.nonzero(kind == k)[0]
        chars[at] = p[rs.randint(0, p.size, at.size)]
    one = off[:256][sizes[:256] == 1]
    chars[one] = np.nonzero(sizes[:256] == 1)[0].astype(np.uint8)
    return off.astype(np.int32), chars


def zipf(n, vocab, g):
    """Token ids with Zipf's frequencies, the frequent ones spread over the vocabulary."""
    p = 1.0 / (torch.arange(vocab, device=DEV, dtype=torch.float64) + 2.7)
    c = torch.cumsum(p, 0)
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64) * c[-1]
    rank = torch.searchsorted(c, u).clamp_(max=vocab - 1)
    return torch.randperm(vocab, generator=g, device=DEV)[rank]


def seen_ids(n, vocab):
    """How many ids of `vocab` are expected among n drawn by zipf()."""
    p = 1.0 / (np.arange(vocab) + 2.7)
    p /= p.sum()
    return float(-np.expm1(n * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def words_of(vocab):
    return -(-vocab // 128) * 4  # 32 tokens a word, rows of whole 16 bytes


# --------------------------------------------------------- prepare
def grammar_inputs(dfa, vocab, mean, seed):
    table, n_states, start, invalid, accept = ROWS[dfa]()
    off, chars = vocabulary(vocab, mean, np.random.RandomState(seed & 0x7FFFFFFF))
    s = {"rows": torch.from_numpy(table).to(DEV), "n_states": n_states, "start": start,
         "invalid": invalid, "accept": accept, "end": vocab - 1, "vocab": vocab,
         "offsets": torch.from_numpy(off).to(DEV), "chars": torch.from_numpy(chars).to(DEV)}
    if own:
        import dfa_parsing_delimiter_gb300 as pp
        s["desc"] = pp.desc_csv() if dfa == "csv" else pp.desc_json_lexer()
    return s


def compiled(dfa, vocab, seed):
    """A vocabulary's vectors and masks, as a program keeps them."""
    s = grammar_inputs(dfa, vocab, 5, seed)
    vectors, allowed = vocab_plain(s)
    s.update(vectors=vectors, allowed=allowed)
    if own:
        import dfa_parsing_delimiter_gb300 as pp
        s["grammar"] = pp.Grammar(vectors, allowed, vocab, s["desc"])
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "vocab":
        s = grammar_inputs(case["dfa"], case["vocab"], case["mean"], seed)
    elif op == "states":
        s = compiled(case["dfa"], case["vocab"], seed)
        rows, cols = case["rows"], case["cols"]
        # mostly tokens that a text goes on with, some that end it
        sound = s["vectors"] >> (4 * (4 if case["dfa"] == "json" else 1)) & 15
        good = torch.nonzero(sound != s["invalid"]).flatten()
        pick = good[zipf(rows * cols, good.numel(), g)]
        wild = torch.randint(0, case["vocab"], (rows * cols,), generator=g, device=DEV)
        odd = torch.rand(rows * cols, generator=g, device=DEV) < 2e-5
        s["tokens"] = torch.where(odd, wild, pick).view(rows, cols).to(torch.int32)
        begin = torch.tensor([4, 3, 4, 9] if case["dfa"] == "json" else [0, 1, 2, 0], device=DEV)
        s["begin"] = begin[torch.randint(0, 4, (rows,), generator=g, device=DEV)].to(torch.uint8)
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.randint(0, cols + 1, (rows,), generator=g, device=DEV).to(torch.int32)
    elif op == "logits":
        s = compiled(case["dfa"], case["vocab"], seed)
        rows, vocab, hist = case["rows"], case["vocab"], case["history"]
        x = torch.randn(rows, vocab, generator=g, device=DEV, dtype=torch.float32).mul_(3.0)
        s["logits"] = x.to(FLOAT[case["type"]])
        s["history"] = zipf(rows * hist, vocab, g).view(rows, hist).to(torch.int32)
        s["history_len"] = torch.randint(hist // 2, hist + 1, (rows,), generator=g, device=DEV).to(torch.int32)
        s["prompt_len"] = (s["history_len"] * torch.rand(rows, generator=g, device=DEV)).to(torch.int32)
        s["repetition"] = 1.0 + 0.3 * torch.rand(rows, generator=g, device=DEV)
        s["presence"] = 0.5 * torch.rand(rows, generator=g, device=DEV)
        s["frequency"] = 0.3 * torch.rand(rows, generator=g, device=DEV)
        count = torch.randint(0, case["bias"] + 1, (rows,), generator=g, device=DEV)
        s["bias_offsets"] = torch.nn.functional.pad(count.cumsum(0), (1, 0)).to(torch.int32)
        total = int(count.sum())
        s["bias_tokens"] = torch.randint(0, vocab, (total,), generator=g, device=DEV).to(torch.int32)
        # an entry names a token that no other entry of its row names
        row = torch.repeat_interleave(torch.arange(rows, device=DEV), count)
        nth = torch.arange(total, device=DEV) - s["bias_offsets"][row].long()
        s["bias_tokens"] = ((s["bias_tokens"][s["bias_offsets"][row].long()].long() + nth * 37) % vocab).to(torch.int32) \
            if vocab > 37 * case["bias"] else (nth % vocab).to(torch.int32)
        s["bias_values"] = torch.randn(total, generator=g, device=DEV) * 4
        begin = torch.tensor([4, 0, 9, 4] if case["dfa"] == "json" else [0, 1, 2, 3], device=DEV)
        s["states"] = begin[torch.randint(0, 4, (rows,), generator=g, device=DEV)].to(torch.uint8)
    else:
        vocab, dim, n = case["vocab"], case["dim"], case["n"]
        s = {"scale": math.sqrt(dim), "pad": 0, "vocab": vocab, "out": FLOAT[case["out"]]}
        ids = zipf(n, vocab, g)
        gone = torch.rand(n, generator=g, device=DEV) < 0.03
        s["ids"] = torch.where(gone, torch.zeros_like(ids), ids).to(torch.int32)
        if op == "embed":
            s["table"] = torch.randn(vocab, dim, generator=g, device=DEV).mul_(0.02).to(FLOAT[case["type"]])
        else:
            s["grad"] = torch.randn(n, dim, generator=g, device=DEV).mul_(1e-2).to(FLOAT[case["type"]])
    s["op"] = op
    return s


# --------------------------------------------------------- plain forms
def vocab_plain(s):
    """Per token the state that each state reaches over its bytes (a nibble a
    state) and per state a bit for each token that does not end invalid."""
    off, vocab = s["offsets"].long(), s["vocab"]
    sizes = off[1:] - off[:-1]
    at = torch.repeat_interleave(torch.arange(vocab, device=DEV), sizes)
    place = torch.arange(s["chars"].numel(), device=DEV) - off[at]
    step = s["rows"][s["chars"].long()]  # [bytes, 16]: the map of each byte
    d, most = 1, int(sizes.max())
    while d < most:  # maps composed over twice the distance each time
        joined = torch.gather(step[d:], 1, step[:-d])
        step = torch.cat([step[:d], torch.where((place[d:] >= d)[:, None], joined, step[d:])])
        d *= 2
    same = torch.arange(16, device=DEV).expand(vocab, 16)
    full = torch.where((sizes > 0)[:, None], step[(off[1:] - 1).clamp(min=0)], same)
    shift = torch.arange(0, 64, 4, device=DEV)
    vectors = (full << shift).sum(1)
    fine = (full[:, :s["n_states"]] != s["invalid"]) & (sizes > 0)[:, None]
    fine[:, s["invalid"]] = False
    fine[s["end"]] = False
    fine[s["end"], s["accept"]] = True
    wide = torch.zeros(s["n_states"], words_of(vocab) * 32, dtype=torch.int64, device=DEV)
    wide[:, :vocab] = fine.t()
    bits = (wide.view(s["n_states"], -1, 32) << torch.arange(32, device=DEV)).sum(2)
    return vectors, bits.to(torch.int32)


def states_plain(s):
    """The state before each token of each row and after the last one."""
    rows, cols = s["tokens"].shape
    maps = s["vectors"][s["tokens"].long()][:, :, None] >> torch.arange(0, 64, 4, device=DEV) & 15
    if s["lengths"] is not None:
        gone = torch.arange(cols, device=DEV) >= s["lengths"][:, None]
        maps = torch.where(gone[:, :, None], torch.arange(16, device=DEV), maps)
    d = 1
    while d < cols:
        maps = torch.cat([maps[:, :d], torch.gather(maps[:, d:], 2, maps[:, :-d])], 1)
        d *= 2
    begin = s["begin"].long()
    after = torch.gather(maps, 2, begin[:, None, None].expand(rows, cols, 1))[:, :, 0]
    return torch.cat([begin[:, None], after], 1).to(torch.uint8)


def logits_plain(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    hist = s["history"].long()
    place = torch.arange(hist.shape[1], device=DEV)[None, :]
    there = place < s["history_len"][:, None]
    told = there & (place >= s["prompt_len"][:, None])
    seen = torch.zeros(rows, vocab, device=DEV).scatter_add_(1, hist, there.float()) > 0
    count = torch.zeros(rows, vocab, device=DEV).scatter_add_(1, hist, told.float())
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    row = torch.repeat_interleave(torch.arange(rows, device=DEV), torch.diff(s["bias_offsets"].long()))
    bias = torch.zeros(rows, vocab, device=DEV)
    bias[row, s["bias_tokens"].long()] = s["bias_values"]
    x = x + bias
    words = s["allowed"][s["states"].long()]
    fine = (words[:, :, None] >> torch.arange(32, dtype=torch.int32, device=DEV) & 1).view(rows, -1)[:, :vocab]
    return torch.where(fine > 0, x, -math.inf).to(s["logits"].dtype)


def embed_plain(s):
    ids = s["ids"].long()
    rows = s["table"][ids].float() * s["scale"]
    return torch.where((ids != s["pad"])[:, None], rows, 0.0).to(s["out"])


def grad_plain(s):
    ids = s["ids"].long()
    g = torch.where((ids != s["pad"])[:, None], s["grad"].float(), 0.0)
    full = torch.zeros(s["vocab"], g.shape[1], device=DEV).index_add_(0, ids, g)
    return (full * s["scale"]).to(s["out"])


def run(s):
    op = s["op"]
    if not own:
        return {"vocab": vocab_plain, "states": states_plain, "logits": logits_plain, "embed": embed_plain,
                "grad": grad_plain}[op](s)
    import dfa_parsing_delimiter_gb300 as pp
    if op == "vocab":
        g = pp.vocab_grammar(s["offsets"], s["chars"], s["desc"], end_id=s["end"])
        return g.vectors, g.allowed
    if op == "states":
        return pp.grammar_states(s["grammar"], s["tokens"], start=s["begin"], lengths=s["lengths"])
    if op == "logits":
        return pp.process_logits(
            s["logits"], history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"],
            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
            bias=(s["bias_offsets"], s["bias_tokens"], s["bias_values"]), grammar=s["grammar"], states=s["states"])
    if op == "embed":
        return pp.embed(s["ids"], s["table"], scale=s["scale"], padding_id=s["pad"], dtype=s["out"])
    return pp.embed_grad(s["ids"], s["grad"], s["vocab"], scale=s["scale"], padding_id=s["pad"], dtype=s["out"])


# --------------------------------------------------------- what a pass needs
def work(case):
    op = case["op"]
    if op == "vocab":
        n_states = 5 if case["dfa"] == "csv" else 16
        v, chars = case["vocab"], case["vocab"] * case["mean"]
        return {"bytes": 4 * (v + 1) + chars + 8 * v + 4 * n_states * words_of(v), "flops": 0}
    if op == "states":
        n = case["rows"] * case["cols"]
        kept = seen_ids(n, case["vocab"])
        return {"bytes": 4 * n + 8 * kept + 2 * case["rows"] + n, "flops": 0}
    if op == "logits":
        n = case["rows"] * case["vocab"]
        masks = min(case["rows"], 4) * words_of(case["vocab"]) * 4
        lists = case["rows"] * (3 * case["history"] + 4 * case["bias"] + 33)  # half of them on average
        return {"bytes": 2 * n * SIZE[case["type"]] + masks + lists, "flops": 2 * n}
    kept = seen_ids(case["n"], case["vocab"])
    if op == "embed":
        size = kept * SIZE[case["type"]] + case["n"] * SIZE[case["out"]]
        return {"bytes": case["dim"] * size + 4 * case["n"], "flops": case["n"] * case["dim"]}
    size = case["n"] * SIZE[case["type"]] + case["vocab"] * SIZE[case["out"]]
    return {"bytes": case["dim"] * size + 4 * case["n"], "flops": case["n"] * case["dim"] + kept * case["dim"]}


# --------------------------------------------------------- 64 bits
def vocab_exact(s):
    """Each token's bytes walked one after the other from every state."""
    table = s["rows"].cpu().numpy()
    off, chars = s["offsets"].cpu().numpy(), s["chars"].cpu().numpy()
    vocab, sizes = s["vocab"], np.diff(off)
    now = np.tile(np.arange(16), (vocab, 1))
    for k in range(int(sizes.max())):
        at = np.nonzero(sizes > k)[0]
        now[at] = np.take_along_axis(table[chars[off[at] + k]], now[at], 1)
    bits = np.zeros((s["n_states"], words_of(vocab) * 32), np.uint8)
    for q in range(s["n_states"]):
        bits[q, :vocab] = (now[:, q] != s["invalid"]) & (sizes > 0) & (q != s["invalid"])
        bits[q, s["end"]] = q in s["accept"]
    vectors = np.zeros(vocab, np.uint64)
    for q in range(16):
        vectors |= now[:, q].astype(np.uint64) << np.uint64(4 * q)
    packed = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
    return vectors.view(np.int64), packed


def states_exact(s):
    tokens, vectors = s["tokens"].cpu().numpy(), s["vectors"].cpu().numpy().view(np.uint64)
    rows, cols = tokens.shape
    size = np.full(rows, cols) if s["lengths"] is None else s["lengths"].cpu().numpy()
    out = np.zeros((rows, cols + 1), np.uint8)
    now = s["begin"].cpu().numpy().copy()
    out[:, 0] = now
    for t in range(cols):
        then = (vectors[tokens[:, t]] >> (4 * now.astype(np.uint64))) & np.uint64(15)
        now = np.where(t < size, then, now).astype(np.uint8)
        out[:, t + 1] = now
    return out


def logits_exact(s):
    """Row by row, over the history's tokens by their counts."""
    x = s["logits"].double().cpu()
    rows, vocab = x.shape
    host = {k: v.cpu().numpy() for k, v in s.items() if isinstance(v, torch.Tensor) and k != "logits"}
    for r in range(rows):
        past, said = int(host["history_len"][r]), int(host["prompt_len"][r])
        tokens = host["history"][r, :past]
        y = x[r].numpy()
        at = np.unique(tokens)
        y[at] = np.where(y[at] > 0, y[at] / np.float64(host["repetition"][r]), y[at] * np.float64(host["repetition"][r]))
        at, n = np.unique(tokens[said:], return_counts=True)
        y[at] -= np.float64(host["frequency"][r]) * n + np.float64(host["presence"][r])
        lo, hi = host["bias_offsets"][r], host["bias_offsets"][r + 1]
        y[host["bias_tokens"][lo:hi]] += host["bias_values"][lo:hi].astype(np.float64)
        mask = np.unpackbits(host["allowed"][host["states"][r]].view(np.uint8), bitorder="little")[:vocab]
        y[mask == 0] = -np.inf
    return x


def embed_exact(s):
    ids = s["ids"].long()
    out = torch.index_select(s["table"], 0, ids).double().mul_(s["scale"])
    out[ids == s["pad"]] = 0
    return out


def grad_exact(s):
    """Rows in the order of their ids, and differences of their running sums."""
    ids, order = torch.sort(s["ids"].long(), stable=True)
    fresh = torch.ones_like(ids, dtype=torch.bool)
    fresh[1:] = ids[1:] != ids[:-1]
    first = torch.nonzero(fresh).flatten()
    last = torch.cat([first[1:], torch.tensor([ids.numel()], device=ids.device)]) - 1
    out = torch.zeros(s["vocab"], s["grad"].shape[1], dtype=torch.float64, device=DEV)
    for lo in range(0, out.shape[1], 256):
        part = s["grad"][:, lo:lo + 256].double()[order]
        sums = part.cumsum(0)
        total = sums[last] - sums[first] + part[first]
        out[ids[first], lo:lo + 256] = total * s["scale"]
    out[s["pad"]] = 0
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"vocab": vocab_exact, "states": states_exact, "logits": logits_exact, "embed": embed_exact,
            "grad": grad_exact}[case["op"]](s)
