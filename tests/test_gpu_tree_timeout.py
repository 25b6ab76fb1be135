"""The bounded waits of the tree attention (skv_set_wait_limit): a limit that is
shorter than what a block's warps wait for ends the call with
SKV_ERR_TIMEOUT, whichever wait runs out first, and the next call on the same
context, store and workspace gives the same bits as before."""
import pytest
import torch

from long_context_decode_ada_b200 import skv
from test_gpu_tree import compare, drafts, make_store

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,kw", [(12, {}), (40, {}), (20, dict(softcap=30.0))])   # 48, 160, 80 rows
def test_short_limits_time_out_and_the_next_call_is_right(N, kw):
    cache, _ = make_store([3000, 700, 40], 2, 4, 64, seed=83)
    q, k, v, _ = drafts(3, N, 2, 4, 47)
    ws = cache.tree_workspace(N, 8)
    want = cache.tree_attention(q, k, v, workspace=ws, **kw)
    compare(cache, want, q, k=k, v=v, **kw)
    try:
        for limit in (1, 64, 500, 1000, 2000, 4000, 8000, 16000, 32000):
            cache.ctx.set_wait_limit(limit)
            out, _ = cache.tree_attention(q, k, v, workspace=ws, **kw)
            if limit <= 64:
                with pytest.raises(skv.SkvError) as e:
                    cache.check()
                assert e.value.code == skv.SKV_ERR_TIMEOUT
                continue
            try:       # (a longer one may be enough)
                cache.check()
                assert torch.equal(out, want[0])
            except skv.SkvError as e:
                assert e.code == skv.SKV_ERR_TIMEOUT
    finally:
        cache.ctx.set_wait_limit(0)
    for _ in range(3):
        out, _ = cache.tree_attention(q, k, v, workspace=ws, **kw)
        cache.check()
        assert torch.equal(out, want[0])


def test_a_limit_that_is_long_enough_changes_nothing():
    cache, _ = make_store([2000], 2, 4, 16, seed=89)
    q, k, v, _ = drafts(1, 24, 2, 4, 49)
    want, _ = cache.tree_attention(q, k, v)
    cache.ctx.set_wait_limit(1_000_000_000)
    out, _ = cache.tree_attention(q, k, v)
    cache.check()
    assert torch.equal(out, want)
    cache.ctx.set_wait_limit(0)
