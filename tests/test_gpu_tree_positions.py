"""Biased scores where the row map leaves resident rows without a position: the
row is reported and skipped, whatever the workspace held before."""
import numpy as np
import pytest
import torch

from long_context_decode_ada_b200 import skv
from _store64 import tree_reference
from test_gpu_tree import drafts, make_store

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,G", [(1, 4), (2, 4), (6, 4), (20, 4), (40, 4)])
@pytest.mark.parametrize("stale", [False, True])
def test_rows_without_a_position(N, G, stale):
    lens = [300, 90]
    cache, dev = make_store(lens, 1, G, 16, f=(0.2, 0.4, 0.4), seed=73)
    q, k, v, _ = drafts(2, N, 1, G, 41)
    slopes = torch.tensor([2.0 ** -(i + 3) for i in range(G)], device="cuda")
    q_pos = (dev["seq_lens"][:, None] + torch.arange(N, device="cuda")[None]).to(torch.int32)
    kw = dict(slopes=slopes, q_pos=q_pos)
    tier = cache.tier.cpu()
    if stale:                       # the lengths of five tokens ago
        seq = dev["seq_lens"] - 5
        lost = [(b, t) for b in range(2) for t in range(lens[b] - 5, lens[b])]
    else:
        seq = dev["seq_lens"]
        lost = [(0, 3), (0, 17), (0, 250), (1, 0), (1, 60)]
        for b, t in lost:
            cache.row_of[b, 0, t] = -1
    assert any(tier[b, 0, t] < 3 for b, t in lost)
    lse = torch.empty((2, N, G), device="cuda")
    outs = []
    for junk in (0x00, 0x3F, 0xFF):
        ws = cache.tree_workspace(N, G, positions=True)
        ws.fill_(junk)
        out, _ = cache.tree_attention(q, k, v, seq_lens=seq, lse=lse, workspace=ws, **kw)
        outs.append((out, lse.clone()))
        with pytest.raises(skv.SkvError) as e:
            cache.check()
        assert e.value.code == skv.SKV_ERR_CORRUPT
    for out, x in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(x, outs[0][1])
    # the tokens that are left, in 64 bits
    if stale:
        for b, t in lost:
            cache.row_of[b, 0, t] = -1
    left = _Left(cache)
    ref = {x: y.cpu() for x, y in dict(k=k, v=v, **kw).items()}
    o, l, ob, lb = left.reference(q.cpu(), **ref)
    out, x = outs[0]
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= ob)
    assert np.all(np.abs(x.double().cpu().numpy() - l) <= lb)


class _Left:
    """tree_reference over the rows of a store that have a position."""

    def __init__(self, cache):
        self.cache = cache

    def reference(self, q, **kw):
        import _store64
        read = _store64.read_store

        def rows(cache, *a):
            units = read(cache, *a)
            for u in units:
                has = u["pos"] >= 0
                for n in ("K", "V", "tier", "row", "pos"):
                    u[n] = u[n][has]
            return units

        _store64.read_store = rows
        try:
            return tree_reference(self.cache, q, **kw)
        finally:
            _store64.read_store = read


def test_every_row_named_is_no_error():
    lens = [500, 0, 77]
    cache, dev = make_store(lens, 2, 2, 32, seed=79)
    for N in (1, 5, 40):
        q, k, v, _ = drafts(3, N, 2, 2, 43)
        q_pos = (dev["seq_lens"][:, None] + torch.arange(N, device="cuda")[None]).to(torch.int32)
        slopes = torch.full((4,), 0.01, device="cuda")
        cache.tree_attention(q, k, v, slopes=slopes, q_pos=q_pos, seq_lens=dev["seq_lens"])
        cache.check()
