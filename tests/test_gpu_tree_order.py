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
