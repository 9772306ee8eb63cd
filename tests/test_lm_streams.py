"""On which stream the binding's own copies run."""
import contextlib

import numpy as np
import pytest
import torch
from torch.overrides import TorchFunctionMode

import dfa_parsing_delimiter_gb300 as pp
import lm_ref as R


class Calls(TorchFunctionMode):
    """Notes each call of torch that may copy, and whether `inside` was set."""

    def __init__(self):
        super().__init__()
        self.inside, self.seen = False, []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        name = getattr(func, "__name__", "")
        if name in ("reshape", "contiguous", "clone", "flatten", "copy_", "empty"):
            self.seen.append((name, self.inside))
        return func(*args, **(kwargs or {}))


def test_embed_grad_flattens_a_gradient_on_the_given_stream(monkeypatch):
    """A sliced [batch, time, width] gradient has no flat view, so it is
    copied: on the stream that reads the copy, from whose memory it comes."""
    calls, given = Calls(), []

    @contextlib.contextmanager
    def on(stream):
        given.append(stream)
        calls.inside = True
        yield
        calls.inside = False

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(pp.lm, "_call", lambda *a: None)
    stream, ids = object(), torch.zeros(3, 4, dtype=torch.int64)
    with calls:
        pp.embed_grad(ids, torch.zeros(3, 5, 8)[:, :-1], 9, stream=stream)
    assert given and all(s is stream for s in given)
    assert calls.seen and all(inside for _, inside in calls.seen), calls.seen


@pytest.mark.gpu
def test_embed_grad_of_a_sliced_gradient_on_another_stream():
    """While the current stream is busy: a copy there would come too late."""
    rng = np.random.default_rng(3)
    batch, time, dim, vocab = 6, 700, 24, 50
    ids = torch.from_numpy(rng.integers(0, vocab, (batch, time))).cuda()
    whole = torch.from_numpy(rng.normal(0, 1, (batch, time + 1, dim))).float().cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.zeros(1 << 28, device="cuda")
    for _ in range(20):
        busy.add_(1)
    got = pp.embed_grad(ids, whole[:, :-1], vocab, stream=s)
    s.synchronize()
    host = got.cpu()
    torch.cuda.synchronize()
    ref, error = R.embed_grad(ids.cpu().numpy().ravel(), whole[:, :-1].reshape(-1, dim).double().cpu().numpy(), vocab, 1, -1)
    R.check(host, ref, error, torch.float32)
