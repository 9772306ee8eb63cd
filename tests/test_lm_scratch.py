"""Where the embedding gradient's scratch comes from, and how much it is."""
import numpy as np
import pytest
import torch

import dfa_parsing_delimiter_gb300 as pp

BIG = (1 << 31) - 65536


def test_sizes():
    size = pp.lib().pp_embed_grad_scratch
    for n, vocab, dim in ((0, 9, 8), (384, 9, 8), (385, 0, 8), (385, 9, 0), (BIG, 9, 8), (385, 9, BIG)):
        assert size(n, vocab, dim) == 0
    for n in (385, 1000, 65536, 65537, 131072, 131073, 1 << 20):
        for dim in (1, 64, 2048):
            assert 8 * n <= size(n, 9, dim)


def test_refusals_need_no_gpu():
    L = pp.lib()
    need = L.pp_embed_grad_scratch(1000, 4, 8)

    def call(n=1000, scratch=32, size=need, out=32):
        return L.pp_embed_grad_noalloc(16, 2, 1, n, 16, 0, 8, 4, 8, 1.0, -1, 0, out, 0, 8, scratch, size, None)

    assert need > 0
    for bad in (dict(scratch=None), dict(size=need - 1), dict(size=0), dict(scratch=40), dict(out=None)):
        assert call(**bad) == pp.PP_EINVAL, bad
    assert call(n=BIG) == pp.PP_ETOOLARGE


@pytest.mark.gpu
@pytest.mark.parametrize("n,dim", [(131072, 2048), (300000, 1024)])
def test_the_call_keeps_no_memory(n, dim):
    """The scratch is torch's, so torch can reuse it and give it back."""
    ids = torch.arange(n, device="cuda") % 1000
    grad = torch.ones(n, dim, device="cuda", dtype=torch.bfloat16)
    pp.embed_grad(ids[:1000], grad[:1000], 1000)  # what a first call sets up
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    out = pp.embed_grad(ids, grad, 1000)
    assert float(out[0, 0]) == (n + 999) // 1000
    del out
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert torch.cuda.mem_get_info()[0] >= free - (32 << 20)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [384, 385, 5000, 131073])
def test_both_entry_points_agree_and_stay_inside_the_scratch(n):
    rng = np.random.default_rng(n)
    vocab, dim = 300, 40
    L, s = pp.lib(), torch.cuda.current_stream().cuda_stream
    ids = torch.from_numpy(rng.integers(-1, vocab + 1, n)).cuda()
    grad = torch.from_numpy(rng.normal(0, 1, (n, dim))).float().cuda()
    need = L.pp_embed_grad_scratch(n, vocab, dim)
    room = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    a, b = torch.empty(2, vocab, dim, device="cuda")
    args = (ids.data_ptr(), 3, 1, n, grad.data_ptr(), 0, dim, vocab, dim, 1.5, 3, 0)
    assert L.pp_embed_grad(*args, a.data_ptr(), 0, dim, s) == pp.PP_OK
    assert L.pp_embed_grad_noalloc(*args, b.data_ptr(), 0, dim, room[256:].data_ptr(), need, s) == pp.PP_OK
    assert torch.equal(a, b) and torch.equal(a, pp.embed_grad(ids, grad, vocab, 1.5, 3))
    assert (room[:256] == 77).all() and (room[256 + need:] == 77).all()


@pytest.mark.parametrize("n", [385, 386, 1000, 4096, 65536, 65537, 131072, 131073, 1 << 20, 3000001])
@pytest.mark.parametrize("dim", [1, 7, 8, 9, 256, 257, 2048])
def test_no_more_than_the_header_states(n, dim):
    """Partial sums 8 ceil(n / L) dim' with L = 32 where that many chunks fill
    the machine, and 8 at the least; the sorted list 8 bytes an id, or from
    65537 ids on 16 and 2 KiB for every 4096 begun; 8 bytes a chunk; 4 KiB."""
    size = pp.lib().pp_embed_grad_scratch(n, 9, dim)
    least = 32 if n // 32 * ((dim + 255) // 256) >= 3648 else 8
    chunks, width = -(-n // least), -(-dim // 8) * 8
    assert size <= 8 * chunks * width + (8 * n if n <= 65536 else 16 * n + 2048 * -(-n // 4096)) + 8 * chunks + 4096
    assert size >= 8 * -(-n // 32) * width + 8 * n
