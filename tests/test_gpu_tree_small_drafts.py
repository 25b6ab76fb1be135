"""Drafted values far below and above unit size: they keep their precision (a
result is linear in them), alone and beside a store, in every form."""
import pytest
import torch

from long_context_decode_ada_b200 import skv
from long_context_decode_ada_b200 import workloads as wl
from test_gpu_tree import compare, drafts, make_store

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 6, 8, 12, 20, 32, 40, 64]      # times 4 heads: 4 to 256 rows a kv head


def some_mask(N, seed):
    g = torch.Generator().manual_seed(seed)
    m = [[(1 << i) | int(torch.randint(0, 1 << min(i, 30), (1,), generator=g)) if i else 1
          for i in range(N)]]
    m = [[x - (1 << 64) if x >> 63 else x for x in row] for row in m]
    return torch.tensor(m, dtype=torch.int64)


@pytest.mark.parametrize("N", ROWS)
@pytest.mark.parametrize("down", [4, 10, 20, 30, 50])
def test_drafted_values_alone(N, down):
    # nothing resident: 2^down times the result is the result of 2^down times the values
    cache, _ = make_store([1], 1, 4, 16, f=(0, 0, 0), seed=93)
    q, k, v, _ = drafts(1, N, 1, 4, 53, torch.bfloat16, torch.bfloat16)
    mask = some_mask(N, N)
    out, _ = cache.tree_attention(q, k, v * 2.0 ** -down, mask=mask.cuda())
    compare(cache, (out.double() * 2.0 ** down, None), q, k=k, v=v, mask=mask)


@pytest.mark.parametrize("N", ROWS)
@pytest.mark.parametrize("down", [0, 7, 12, 24])
@pytest.mark.parametrize("lens", [[64], [700], [1500]])
def test_beside_a_store(N, down, lens):
    # values of the store of unit size, the drafted ones smaller
    cache, _ = make_store(lens, 1, 4, 16, seed=95)
    q, k, v, _ = drafts(1, N, 1, 4, 55, torch.bfloat16, torch.bfloat16)
    v = v * 2.0 ** -down
    mask = some_mask(N, N)
    for splits in (1, 0):
        got = cache.tree_attention(q, k, v, mask=mask.cuda(), num_splits=splits)
        compare(cache, got, q, k=k, v=v, mask=mask)


@pytest.mark.parametrize("N", ROWS)
def test_small_values_everywhere(N):
    lens = [600]
    w = wl.custom(97, 1, 1, 4, 16, lens, wl.MODE_QUOTA, quota=[[100, 200, 200]], scatter=True)
    w.V = (w.V.float() * 2.0 ** -10).half()
    dev = skv.workload_to_device(w)
    cache = skv.build_cache(skv.Context(16), w, dev)
    q, k, v, _ = drafts(1, N, 1, 4, 57, torch.bfloat16, torch.bfloat16)
    v = v * 2.0 ** -10
    for splits in (1, 3):
        got = cache.tree_attention(q, k, v, num_splits=splits)
        compare(cache, got, q, k=k, v=v)


@pytest.mark.parametrize("N", [2, 6, 12, 20, 40])
def test_small_values_beside_ones_beyond_fp16(N):
    # one token's values are beyond fp16, all the others' tiny
    cache, _ = make_store([1], 1, 4, 16, f=(0, 0, 0), seed=99)
    q, k, v, _ = drafts(1, N, 1, 4, 59, torch.bfloat16, torch.bfloat16)
    v = v * 2.0 ** -20
    mask = torch.full((1, N), (1 << N) - 2, dtype=torch.int64)
    mask[0, N - 1] = (1 << N) - 1
    clean, _ = cache.tree_attention(q, k, v, mask=mask.cuda())
    v[0, 0] = 1e6
    out, _ = cache.tree_attention(q, k, v, mask=mask.cuda())
    assert torch.equal(out[:, :N - 1], clean[:, :N - 1])
    compare(cache, (out, None), q, k=k, v=v, mask=mask)
