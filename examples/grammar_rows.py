"""A toy language model that learns rows of a table and answers with rows that
parse: the operators of a language model beside the parser they belong to.

  1. the vocabulary is a CSV file; pp.parse_csv reads its pieces into a string
     column, and pp.vocab_grammar puts that column under the CSV DFA;
  2. the training rows' pieces become ids, pp.embed looks them up, and its
     gradient (pp.embed_grad, through autograd) trains the table by
     pp.adamw_step;
  3. the model answers a few pieces at a time: a table of which piece follows
     which drafts some, pp.grammar_states gives each row's DFA state before
     each of them, pp.process_logits applies penalties, a bias and the
     grammar's mask to the model's logits at all of them, pp.token_probs makes
     probabilities of those, and pp.verify_drafts accepts drafts by them and
     draws the piece that follows;
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
    state = pp.adamw_state([table, head])
    losses = []
    for _ in range(steps):
        table.grad = head.grad = None
        logits = pp.embed(ids, table, scale=dim ** 0.5 / 4) @ head
        loss = torch.nn.functional.cross_entropy(logits, targets)
        loss.backward()
        pp.adamw_step([table, head], None, state, lr=0.05, weight_decay=0.0)
        losses.append(loss.detach())
    return table.detach(), head.detach(), torch.stack(losses).tolist()


def following(ids, vocab: int):
    """How likely each piece is after each, by counting: what drafts are drawn from."""
    count = torch.full((vocab * vocab,), 0.05, device=ids.device)
    pairs = ids[:-1].long() * vocab + ids[1:].long()
    count.index_add_(0, pairs, torch.ones(pairs.numel(), device=ids.device))
    count = count.view(vocab, vocab)
    return count / count.sum(1, keepdim=True)


def answer(table, head, grammar, after, rows: int, length: int, drafted: int, generator):
    """`rows` answers of about `length` pieces at most; (pieces, their states,
    which are over, how many rounds it took)."""
    device, dim = table.device, table.size(1)
    end, k = PIECES.index("<end>"), drafted
    said = torch.full((rows, length + k + 2), end, dtype=torch.int32, device=device)
    said[:, 0] = PIECES.index("\n")  # what a row begins after
    n = torch.ones(rows, dtype=torch.int32, device=device)  # pieces so far; the first was given
    states = torch.full((rows,), grammar.start_state, dtype=torch.uint8, device=device)
    over = torch.zeros(rows, dtype=torch.bool, device=device)
    place = torch.arange(k + 1, dtype=torch.int32, device=device)
    each = rows * (k + 1)  # a row of logits for each draft and one more
    of_row = torch.arange(rows, dtype=torch.int32, device=device).repeat_interleave(k + 1)
    one = torch.arange(each + 1, dtype=torch.int32, device=device)
    ones = torch.ones(each, device=device)
    for rounds in range(1, length + 1):
        last = said.gather(1, n[:, None].long() - 1)
        line, probs = [last], []
        for _ in range(k):
            probs.append(after[line[-1][:, 0].long()])
            line.append(torch.multinomial(probs[-1], 1, generator=generator).to(torch.int32))
        line = torch.cat(line, 1)
        drafts = line[:, 1:].contiguous()
        logits = (pp.embed(line, table, scale=dim ** 0.5 / 4) @ head).view(each, -1)
        so_far = (n[:, None] + place).flatten()
        # the text may end after a row; the end gets likelier as time runs out
        bias = (one, torch.full((each,), end, dtype=torch.int32, device=device),
                torch.where(so_far <= length // 2, -2.0, 20.0))
        before = pp.grammar_states(grammar, drafts, start=states)
        logits = pp.process_logits(logits, history=said.scatter(1, (n[:, None] + place[:k]).long(), drafts), history_row=of_row,
                                   history_len=so_far, prompt_len=torch.ones_like(so_far), repetition=1.05 * ones,
                                   presence=0.05 * ones, frequency=0.02 * ones, bias=bias, grammar=grammar,
                                   states=before.flatten())
        target = pp.token_probs(logits)
        tokens, counts = pp.verify_drafts(target, drafts, torch.rand(rows, k, generator=generator, device=device),
                                          torch.rand(rows, generator=generator, device=device),
                                          draft_probs=torch.stack(probs, 1).flatten(0, 1) if k else None)
        # an answer ends with its end, and at its full length
        ends = (tokens == end) & (place < counts[:, None])
        counts = torch.where(ends.any(1), torch.minimum(counts, ends.int().argmax(1).to(torch.int32) + 1), counts)
        counts = torch.where(over | (n > length), 0, counts)
        at = (n[:, None] + place).long().clamp(max=said.size(1) - 1)
        said.scatter_(1, at, torch.where(place < counts[:, None], tokens, said.gather(1, at)))
        states = pp.grammar_states(grammar, tokens, start=states, lengths=counts)[:, -1]
        over |= (ends & (place < counts[:, None])).any(1)
        n += counts
        if bool((over | (n > length)).all()):
            break
    return said[:, 1:], states, over, rounds


def run(device="cuda", seed: int = 0, rows: int = 8, length: int = 48, steps: int = 60, drafted: int = 3) -> dict:
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
    pieces, states, over, rounds = answer(table, head, grammar, following(ids, len(PIECES)), rows, length, drafted, g)
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
    return dict(losses=losses, texts=texts, parsed=parsed, over=over.tolist(), same_states=torch.equal(states, again),
                rounds=rounds, said=int((pieces != end).sum()))


if __name__ == "__main__":
    out = run()
    print("loss %.3f -> %.3f; %d pieces in %d rounds" % (out["losses"][0], out["losses"][-1], out["said"], out["rounds"]))
    for t, p in zip(out["texts"], out["parsed"]):
        print(repr(t), "->", "unfinished" if p is None else "%d records, error bits %d" % (p["n_records"], p["error"]))
