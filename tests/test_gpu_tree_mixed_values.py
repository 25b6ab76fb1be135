"""Tree attention where dense, coded and drafted values of different sizes meet
in one sum: the weights of each keep their precision."""
import math

import pytest
import torch

from long_context_decode_ada_b200 import skv
from long_context_decode_ada_b200 import workloads as wl
from test_gpu_tree import compare, drafts, make_store

pytestmark = pytest.mark.gpu

T = 40000


@pytest.mark.parametrize("size", [1e-3, 1e-2, 1.0, 3000.0])
@pytest.mark.parametrize("G,N", [(4, 1), (4, 4), (4, 8), (4, 12)])
def test_dense_rows_before_coded_ones(size, G, N):
    # the first 192 tokens dense, a heavy one in each 16 of them; then coded tokens
    # of weights of 2^-12 that carry almost half of the sum, values of one sign
    g = torch.Generator().manual_seed(71)
    q = (1 + 0.3 * torch.randn((1, N, G, 128), generator=g)).half().cuda()
    w = wl.custom(113, 1, 1, G, 64, [T], wl.MODE_QUOTA, quota=[[192, 20000, T - 20192]], scatter=True,
                  k_scale=0.1)
    w.utility[0, 0, :192] = 10.0
    w.V = ((1 + 0.25 * w.V.float()) * size).to(torch.float16)
    m = q.float().cpu().mean((0, 1, 2))
    s = (q.float().cpu() @ m).mean()
    w.K[0, 0, 5:192:16] = (m * (8.3 * math.sqrt(128) / s)).to(torch.float16)
    dev = skv.workload_to_device(w)
    cache = skv.build_cache(skv.Context(64), w, dev)
    cache.check()
    assert torch.all(cache.tier[0, 0, :192] == 0)
    lse = torch.empty((1, N, G), device="cuda")
    for splits in (1, 0):
        got = cache.tree_attention(q, lse=lse, num_splits=splits)
        compare(cache, got, q)


@pytest.mark.parametrize("f", [(1, 0, 0), (0, 0.5, 0.5), (0.2, 0.4, 0.3)])
@pytest.mark.parametrize("down", [2, 5, 8, 11])
@pytest.mark.parametrize("G,N", [(1, 4), (1, 31), (4, 8), (4, 20)])
def test_small_drafts_beside_a_store_far_away(f, down, G, N):
    # a store of unit values that the bias takes nearly all weight from: what the
    # results are made of is drafted values 2^down times smaller
    lens = [100, 17]
    cache, dev = make_store(lens, 1, G, 16, f=f, seed=127)
    q, k, v, _ = drafts(2, N, 1, G, 73, torch.bfloat16, torch.bfloat16)
    v = v * 2.0 ** -down
    g = torch.Generator().manual_seed(N)
    q_pos = (dev["seq_lens"].cpu()[:, None] + torch.randint(20, 50, (2, N), generator=g)).to(torch.int32)
    kw = dict(slopes=torch.full((G,), 0.7, device="cuda"), q_pos=q_pos.cuda())
    lse = torch.empty((2, N, G), device="cuda")
    for splits in (1, 3):
        got = cache.tree_attention(q, k, v, lse=lse, seq_lens=dev["seq_lens"], num_splits=splits, **kw)
        compare(cache, got, q, k=k, v=v, **kw)


def test_drafts_of_a_thousandth_beside_heavier_dense_values():
    # weights of the store of 2^-10 and less, its values 32 times the drafted
    # ones: found by random calls, 1.4 times the bound
    lens = [100, 64]
    w = wl.custom(2019, 2, 1, 1, 16, lens, wl.MODE_QUOTA, quota=[[t, 0, 0] for t in lens], scatter=True)
    w.V = (w.V.float() * 2.0 ** -7).half()
    dev = skv.workload_to_device(w)
    cache = skv.build_cache(skv.Context(16), w, dev)
    for seed in range(24):
        N = 20 + seed % 12
        q, k, v, _ = drafts(2, N, 1, 1, seed, torch.bfloat16, torch.bfloat16)
        v = v * 2.0 ** -12
        g = torch.Generator().manual_seed(seed)
        q_pos = (dev["seq_lens"].cpu()[:, None] + torch.randint(0, N, (2, N), generator=g)).to(torch.int32)
        kw = dict(slopes=torch.full((1,), 0.5, device="cuda"), q_pos=q_pos.cuda())
        for splits in (1, 3):
            got = cache.tree_attention(q, k, v, seq_lens=dev["seq_lens"], num_splits=splits, **kw)
            compare(cache, got, q, k=k, v=v, **kw)
