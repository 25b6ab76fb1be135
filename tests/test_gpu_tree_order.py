"""Tree attention where one unit follows another in a run: what a unit leaves in
shared memory (query fragments, sums, flags) never reaches the next one's
results.  Units short enough that nothing but the kernels' own barriers and
waits keeps them apart."""
import pytest
import torch

from test_gpu_tree import compare, drafts, make_store

pytestmark = pytest.mark.gpu


def unlike_queries(q):
    """Every sequence's queries at another size: one unit's in place of another's
    would change the outputs by far more than any bound."""
    size = 2.0 ** (torch.arange(q.shape[0]) % 5 - 2)
    return (q.float() * size.view(-1, 1, 1, 1).cuda()).to(q.dtype)


@pytest.mark.parametrize("G,N", [(1, 8), (4, 2), (2, 8), (4, 4), (4, 8)])
@pytest.mark.parametrize("lens", [[0] * 39 + [2], [1 + b % 3 for b in range(40)],
                                  [17 * (b % 4) for b in range(40)]])
def test_queries_of_the_unit_itself(G, N, lens):
    # up to 8, 16 and 32 rows a kv head; drafted tokens alone, or with one or a
    # few tiles, many units a run
    cache, _ = make_store(lens, 2, G, 16, f=(0.3, 0.3, 0.4), seed=61)
    q, k, v, _ = drafts(len(lens), N, 2, G, 33)
    q = unlike_queries(q)
    lse = torch.empty((len(lens), N, 2 * G), device="cuda")
    for splits in (1, 4):
        got = cache.tree_attention(q, k, v, lse=lse, num_splits=splits)
        compare(cache, got, q, k=k, v=v)


@pytest.mark.parametrize("n", [9, 16, 20, 32])             # 36 to 128 rows a kv head
@pytest.mark.parametrize("drafted", [False, True])
def test_units_of_one_tile_behind_longer_ones(n, drafted):
    # one tile: the second stream has nothing to do in the unit.  Units of more
    # than 128 rows, of several tiles and of other sizes lie between
    lens = [300, 5, 40, 64, 0, 9, 700, 1, 60, 33, 128, 20]
    N = 64 if drafted else n
    cache, _ = make_store(lens, 2, 4, 64, f=(0.0, 0.5, 0.5), seed=71)
    B = len(lens)
    q, k, v, _ = drafts(B, N, 2, 4, 37)
    q = unlike_queries(q)
    count = torch.tensor([N if b % 5 == 0 else n for b in range(B)], dtype=torch.int32)
    kw = dict(k=k, v=v) if drafted else {}
    lse = torch.empty((B, N, 8), device="cuda")
    for splits in (1, 3):
        got = cache.tree_attention(q, count=count.cuda(), lse=lse, num_splits=splits, **kw)
        compare(cache, got, q, count=count, **kw)


@pytest.mark.parametrize("N", [9, 12, 16, 17, 25, 32])     # 36 to 128 rows a kv head
@pytest.mark.parametrize("lens", [[0, 1], [64, 10], [128, 65], [400, 200]])
def test_values_beyond_fp16_that_every_row_sees(N, lens):
    # the drafted tile alone, or behind one or two or more tiles: it falls to
    # either stream, and rows of both write what fp16 does not hold
    cache, _ = make_store(lens, 1, 4, 16, f=(0.0, 0.6, 0.4), seed=67)
    q, k, v, _ = drafts(2, N, 1, 4, 35, torch.bfloat16, torch.bfloat16)
    mask = torch.full((2, N), (1 << N) - 1, dtype=torch.int64)
    v[0, 0, 0, 3], v[0, N - 1, 0, 100], v[1, 1, 0, 77] = 2e6, -4e5, 3e8
    lse = torch.empty((2, N, 4), device="cuda")
    for splits in (1, 2, 0):
        got = cache.tree_attention(q, k, v, mask=mask.cuda(), lse=lse, num_splits=splits)
        compare(cache, got, q, k=k, v=v, mask=mask)
    v[0, 0, 0, 3], v[0, 1, 0, 4] = float("inf"), float("nan")
    out, _ = cache.tree_attention(q, k, v, mask=mask.cuda())
    assert torch.all(out[0, :, :, 3] == float("inf")) and torch.isnan(out[0, :, :, 4]).all()
