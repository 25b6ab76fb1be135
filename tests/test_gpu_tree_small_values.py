"""Tree attention over stores whose values are far from unit size: the weights
keep their precision whatever the value scales are, also beside one token that
takes most of the weight (many weights of 2^-12 that carry half of the sum)."""
import math

import pytest
import torch

from long_context_decode_ada_b200 import skv
from long_context_decode_ada_b200 import workloads as wl
from test_gpu_tree import compare

pytestmark = pytest.mark.gpu


T = 40000


def heavy_store(G, q, size, tier, seed):
    """One kv head of 40000 tokens of one tier.  Values of token t are about
    size(t) (one sign: their sum does not cancel), keys a tenth of the usual
    (weights of 2^-12), but for a token in each of the first 12 times 16 that
    the queries see at about 8.3: whatever takes 16 tokens at a time meets one
    first, and the others carry almost half of the sum."""
    quota = [[T * (tier == x) for x in range(3)]]
    w = wl.custom(seed, 1, 1, G, 64, [T], wl.MODE_QUOTA, quota=quota, scatter=True, k_scale=0.1)
    w.V = ((1 + 0.25 * w.V.float()) * size(torch.arange(T)).view(1, 1, -1, 1)).to(torch.float16).contiguous()
    m = q.float().cpu().mean((0, 1, 2))
    s = (q.float().cpu() @ m).mean()
    w.K[0, 0, 5:192:16] = (m * (8.3 * math.sqrt(128) / s)).to(torch.float16)
    dev = skv.workload_to_device(w)
    cache = skv.build_cache(skv.Context(64), w, dev)
    cache.check()
    return cache


SIZES = {
    "1e-2": lambda t: torch.full_like(t, 1e-2, dtype=torch.float32),
    "1e-3": lambda t: torch.full_like(t, 1e-3, dtype=torch.float32),
    "1e-4": lambda t: torch.full_like(t, 1e-4, dtype=torch.float32),
    "300": lambda t: torch.full_like(t, 300.0, dtype=torch.float32),
    "rising": lambda t: 1e-4 * 10.0 ** (t / 6000.0),
    "falling": lambda t: 1e3 * 10.0 ** (-t / 6000.0),
    "one large": lambda t: torch.where(t == 25000, 2000.0, 1e-3),
}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("tier", [1, 2])
@pytest.mark.parametrize("G,N", [(1, 1), (4, 1), (4, 4), (4, 7), (4, 12)])
def test_small_and_large_values(size, tier, G, N):
    # 1, 4, 16, 28 and 48 rows a kv head; fp16 results; one run, and many
    g = torch.Generator().manual_seed(51)
    q = (1 + 0.3 * torch.randn((1, N, G, 128), generator=g)).half().cuda()
    cache = heavy_store(G, q, SIZES[size], tier, 91)
    lse = torch.empty((1, N, G), device="cuda")
    for splits in (1, 0):
        got = cache.tree_attention(q, lse=lse, num_splits=splits)
        compare(cache, got, q)
