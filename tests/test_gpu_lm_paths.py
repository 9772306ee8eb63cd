"""Paths of the language-model operators that sizes alone decide on: several
tiles a block and several blocks a row of states, and gradients with scratch
in graphs and on streams at once."""
import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp
from test_gpu_lm import dev, grad_ids, make_grammar

pytestmark = pytest.mark.gpu


def walk(to, tokens, start, lengths):
    """States along rows of tokens, column by column; a token outside the vocabulary leads to 255."""
    to = np.concatenate([to, np.zeros((len(to), 16 - to.shape[1]), int)], 1)
    out = np.zeros((tokens.shape[0], tokens.shape[1] + 1), np.uint8)
    out[:, 0] = now = start.astype(int)
    step = np.concatenate([np.pad(to, ((0, 1), (0, 1))), np.full((1, 17), 255)])  # state 16 stands for 255
    step[:, 16] = 255
    step[len(to)] = np.r_[0:16, 255]  # a token past the length: nothing changes
    fine = (tokens >= 0) & (tokens < len(to))
    row = np.where(fine, tokens, len(to) + 1)
    row = np.ascontiguousarray(np.where(np.arange(tokens.shape[1]) < lengths[:, None], row, len(to)).T)
    for t in range(len(row)):
        now = step[row[t], np.minimum(now, 16)]
        out[:, t + 1] = now
    return out


@pytest.mark.parametrize("kind", ["csv", "json", "sixteen", "seven"])
@pytest.mark.parametrize("rows,cols", [(1, 50000), (2, 200001), (320, 6000), (305, 2561), (5, 40961), (40, 20000)])
def test_states_over_tiles_and_blocks(rows, cols, kind):
    """A row's blocks take one tile or several, alone or in clusters; tokens
    outside the vocabulary and lengths fall in the first, a middle and the
    last of them."""
    g, to, desc = make_grammar(kind, n=500, seed=1)
    rng = np.random.default_rng(rows + cols)
    calm = np.nonzero((to != (desc.invalid_state if desc.invalid_state != 255 else -1)).all(1))[0]
    calm = calm if calm.size else np.arange(500)
    cases = []  # tokens, start, lengths
    for at in (None, 0, 700, cols // 2, cols - 1300, cols - 1):
        for size in (cols, cols // 2 + 3, 900, cols - 1)[:4 if rows < 40 else 2]:
            tokens = calm[rng.integers(0, calm.size, (rows, cols))].astype(np.int32)
            if at is not None:
                tokens[::2, at] = rng.choice([-1, 500, 1 << 30], tokens[::2, at].shape)
            start = rng.integers(0, desc.n_states, rows).astype(np.uint8)
            start[rows // 2] = 255 if at == 700 else start[rows // 2]
            lengths = np.full(rows, size, np.int32)
            lengths[1 + rows // 3:] = rng.integers(0, cols + 1, rows - 1 - rows // 3)
            cases.append((tokens, start, lengths))
    want = walk(to, *(np.concatenate(x) for x in zip(*cases))).reshape(len(cases), rows, cols + 1)
    for k, (tokens, start, lengths) in enumerate(cases):
        for dtype in (torch.int32, torch.int64):
            got = pp.grammar_states(g, dev(tokens).to(dtype), start=dev(start), lengths=dev(lengths))
            assert np.array_equal(got.cpu().numpy(), want[k]), k


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [1000, 20000, 140000])
def test_gradients_with_scratch_in_a_graph(n, accumulate):
    """Sort, zeros, sums and joins captured, and replayed with other inputs."""
    rng = np.random.default_rng(n)
    vocab, dim = 3000, 72
    ids, grad = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, dim, device="cuda")
    out = torch.zeros(vocab, dim, device="cuda")

    def step(out):
        return pp.embed_grad(ids, grad, vocab, scale=0.5, padding_id=7, out=out, accumulate=accumulate)

    def fill(how):
        ids.copy_(torch.from_numpy(grad_ids(rng, n, vocab, how)))
        grad.copy_(torch.from_numpy(rng.normal(0, 1, (n, dim))))

    fill("any")
    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for how in ("zipf", "one", "any", "runs", "outside", "zipf"):
        fill(how)
        first = torch.from_numpy(rng.normal(0, 1, (vocab, dim))).float().cuda()
        out.copy_(first)
        graph.replay()
        want = step(first.clone())
        torch.cuda.synchronize()
        assert torch.equal(out, want), how


@pytest.mark.parametrize("n", [900, 30000, 150000])
def test_gradients_on_streams_at_once(n):
    """Each call's scratch is its own, also while others run."""
    rng = np.random.default_rng(n)
    vocab, dim = 2000, 64
    cases = [(dev(grad_ids(rng, n, vocab, how)), torch.randn(n, dim, device="cuda")) for how in ("zipf", "any", "one", "runs")]
    want = [pp.embed_grad(i, g, vocab) for i, g in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for s, (i, g) in zip(streams, cases):
            got.append(pp.embed_grad(i, g, vocab, stream=s))
    torch.cuda.synchronize()
    for k, y in enumerate(got):
        assert torch.equal(y, want[k % len(want)])
