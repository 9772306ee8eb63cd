"""A toy language model that learns rows of a table and answers with rows that
parse: the operators of a language model beside the parser they belong to.

  1. the vocabulary is a CSV file; pp.parse_csv reads its pieces into a string
     column, and pp.vocab_grammar puts that column under the CSV DFA;
  2. the training rows' pieces become ids, pp.embed looks them up, and its
     gradient (pp.embed_grad, through autograd) trains the table;
  3. the model answers piece by piece: pp.process_logits applies penalties,
     a bias and the grammar's mask for each row's DFA state, and
     pp.grammar_states moves the states on;
  4. pp.parse_csv reads the answers back.

Run:  python examples/grammar_rows.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dfa_parsing_delimiter_gb300 as pp  # noqa: E402

PIECES = ["<end>", ",", "\n", '"', "apples", "pears", "plums", "figs", " and ", ", ", "1", "2", "3", "7", "12", "40",
          ".5", ".25", ".00"]


def vocabulary_file() -> bytes:
    """One piece a record, quoted where CSV needs it."""
    def quoted(p):
        return '"' + p.replace('"', '""') + '"' if any(c in p for c in ',\n"') else p
    return "\n".join(quoted(p) for p in PIECES).encode() + b"\n"


def training_rows(n: int, rng) -> list[list[int]]:
    """Rows of a name (sometimes quoted, with a comma in it), a count and a price."""
    at = {p: i for i, p in enumerate(PIECES)}
    rows = []
    for _ in range(n):
        fruit = [at[PIECES[4 + i]] for i in rng.integers(0, 4, 2)]
        name = [fruit[0]] if rng.random() < 0.5 else [at['"'], fruit[0], at[", "], fruit[1], at['"']]
        rows.append(name + [at[","], 10 + int(rng.integers(0, 6)), at[","], 10 + int(rng.integers(0, 6)),
                            16 + int(rng.integers(0, 3)), at["\n"]])
    return rows


def read_vocabulary(device):
    data = np.frombuffer(vocabulary_file(), np.uint8).copy()
    ((offsets, chars),), status = pp.parse_csv(torch.from_numpy(data).to(device), ["str"])
    assert status["error"] == 0 and status["n_records"] == len(PIECES), status
    return offsets, chars


def train(ids, targets, vocab: int, dim: int, steps: int, generator):
    """A bigram model: the next piece from this one's vector."""
    device = ids.device
    table = (torch.randn(vocab, dim, generator=generator, device=device) * 0.3).requires_grad_()
    head = (torch.randn(dim, vocab, generator=generator, device=device) * 0.3).requires_grad_()
    opt = torch.optim.Adam([table, head], lr=0.05)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        logits = pp.embed(ids, table, scale=dim ** 0.5 / 4) @ head
        loss = torch.nn.functional.cross_entropy(logits, targets)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return table.detach(), head.detach(), torch.stack(losses).tolist()


def answer(table, head, grammar, rows: int, length: int, generator):
    """`rows` answers of at most `length` pieces; (pieces, their states)."""
    device, dim, vocab = table.device, table.size(1), table.size(0)
    said = torch.zeros(rows, length + 1, dtype=torch.int32, device=device)
    said[:, 0] = PIECES.index("\n")  # what a row begins after
    states = torch.full((rows,), grammar.start_state, dtype=torch.uint8, device=device)
    over = torch.zeros(rows, dtype=torch.bool, device=device)
    ones = torch.ones(rows, device=device)
    end = PIECES.index("<end>")
    one = torch.arange(rows + 1, dtype=torch.int32, device=device)
    first = torch.ones(rows, dtype=torch.int32, device=device)  # the given part: the first piece
    for t in range(length):
        logits = pp.embed(said[:, t], table, scale=dim ** 0.5 / 4) @ head
        # the text may end after a row; the end gets likelier as time runs out
        bias = (one, torch.full((rows,), end, dtype=torch.int32, device=device),
                torch.full((rows,), -2.0 if t < length // 2 else 20.0, device=device))
        said_so_far = torch.full((rows,), t + 1, dtype=torch.int32, device=device)
        logits = pp.process_logits(logits, history=said, history_len=said_so_far, prompt_len=first,
                                   repetition=1.05 * ones, presence=0.05 * ones, frequency=0.02 * ones, bias=bias,
                                   grammar=grammar, states=states)
        noise = -torch.log(-torch.log(torch.rand(rows, vocab, generator=generator, device=device).clamp(1e-7, 1 - 1e-7)))
        piece = torch.where(over, end, (logits + noise).argmax(1)).to(torch.int32)
        over |= piece == end
        said[:, t + 1] = piece
        states = pp.grammar_states(grammar, piece[:, None], start=states)[:, 1]
    return said[:, 1:], states, over


def run(device="cuda", seed: int = 0, rows: int = 8, length: int = 48, steps: int = 60) -> dict:
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    offsets, chars = read_vocabulary(device)
    end = PIECES.index("<end>")
    grammar = pp.vocab_grammar(offsets, chars, pp.desc_csv(), end_id=end)
    text = [PIECES.index("\n")]
    for row in training_rows(200, rng):
        text += row
    ids = torch.tensor(text, dtype=torch.int32, device=device)
    table, head, losses = train(ids[:-1], ids[1:].long(), len(PIECES), 16, steps, g)
    pieces, states, over = answer(table, head, grammar, rows, length, g)
    # the same states from the whole answers at once
    again = pp.grammar_states(grammar, pieces)[:, -1]
    texts = ["".join(PIECES[i] for i in line if i != end) for line in pieces.tolist()]
    parsed = []
    for t, ok in zip(texts, grammar.accepts(states).tolist()):
        if not ok:
            parsed.append(None)
            continue
        data = torch.from_numpy(np.frombuffer(t.encode(), np.uint8).copy()).to(device)
        parsed.append(pp.parse_csv(data, ["str", "str", "str"])[1])
    return dict(losses=losses, texts=texts, parsed=parsed, over=over.tolist(), same_states=torch.equal(states, again))


if __name__ == "__main__":
    out = run()
    print("loss %.3f -> %.3f" % (out["losses"][0], out["losses"][-1]))
    for t, p in zip(out["texts"], out["parsed"]):
        print(repr(t), "->", "unfinished" if p is None else "%d records, error bits %d" % (p["n_records"], p["error"]))
