"""The stream argument of the tree attention and the eviction: buffers that a
call makes itself (outputs, new stores, cursors, workspaces) are filled and
used in its stream's order, whatever is queued on the current one."""
import pytest
import torch

from long_context_decode_ada_b200 import skv
from test_gpu_evict import check_eviction, kept_reference, scores
from test_gpu_evict import make_store as make_evict_store
from test_gpu_tree import drafts, make_store

pytestmark = pytest.mark.gpu


def busy():
    """Some milliseconds of work on the current stream."""
    x = torch.randn((4096, 4096), device="cuda")
    for _ in range(20):
        x = (x @ x) * 1e-3
    return x


def test_outputs_made_by_the_call():
    cache, _ = make_store([1200, 50], 2, 4, 32, seed=23)
    side = torch.cuda.Stream()
    for N in (2, 6, 20, 40):
        q, k, v, _ = drafts(2, N, 2, 4, 12)
        want, _ = cache.tree_attention(q, k, v)
        torch.cuda.synchronize()
        keep = busy()
        out, _ = cache.tree_attention(q, k, v, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del keep
    cache.check()


def test_workspaces_made_by_the_call():
    # what is made on the current stream while the call's kernels run is no part
    # of their workspace
    cache, _ = make_store([9000, 300], 2, 4, 64, seed=25)
    q, k, v, _ = drafts(2, 12, 2, 4, 13)
    want, _ = cache.tree_attention(q, k, v)
    n = cache.tree_workspace(12, 8).numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append(cache.tree_attention(q, k, v, stream=side)[0])
        for _ in range(4):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    cache.check()


@pytest.mark.parametrize("computed_cursor", [False, True])
def test_stores_made_by_the_call(computed_cursor):
    lens, keep = [700, 300], [200, 100]
    cache, dev = make_evict_store(lens, 2, 1, 16, seed=13)
    s = scores((2, 2, 700), 3).cuda()
    kd = torch.tensor(keep, dtype=torch.int32).cuda()
    if not computed_cursor:
        cache.free_cursor()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = busy()
    new = cache.evict(s, dev["seq_lens"], kd, sink=2, recent=8, stream=side)
    torch.cuda.synchronize()
    want = kept_reference(cache.tier.cpu().numpy(), s.cpu().numpy(), lens, keep, 2, 8)
    check_eviction(cache, new, want, dev)
    del x


@pytest.mark.parametrize("named", [False, True])
def test_a_store_dropped_while_its_eviction_runs(named):
    lens, keep = [3000, 2000], [700, 100]
    cache, dev = make_evict_store(lens, 2, 1, 16, seed=17)
    s = scores((2, 2, 3000), 5).cuda()
    kd = torch.tensor(keep, dtype=torch.int32).cuda()
    first = cache.evict(s, dev["seq_lens"], kd)
    torch.cuda.synchronize()
    want = [getattr(first, n).clone() for n in ("tier", "row_of", "page_indptr")]
    side = torch.cuda.Stream()
    sizes = [cache.tier.numel(), 4 * cache.row_of.numel(), 4 * cache.page_ids.numel()]
    ws = cache._ws_evict.numel()
    with torch.cuda.stream(side):
        x = busy()
    if named:
        cache = cache.evict(s, dev["seq_lens"], kd, stream=side)   # (the old store goes)
    else:
        with torch.cuda.stream(side):
            cache = cache.evict(s, dev["seq_lens"], kd)
    for n in sizes + [ws]:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    cache.check()
    for n, w in zip(("tier", "row_of", "page_indptr"), want):
        assert torch.equal(getattr(cache, n), w), n
    del x


def test_streams_of_another_device_are_refused():
    class Elsewhere:
        device = torch.device("cuda", 7)
        cuda_stream = 0

    cache, dev = make_store([40], 1, 4, 16, seed=1)
    q, k, v, _ = drafts(1, 2, 1, 4, 1)
    with pytest.raises(skv.SkvError) as e:
        cache.tree_attention(q, k, v, stream=Elsewhere())
    assert e.value.code == skv.SKV_ERR_ARG
    with pytest.raises(skv.SkvError) as e:
        cache.evict(torch.zeros((1, 1, 40), device="cuda"), dev["seq_lens"],
                    torch.ones(1, dtype=torch.int32, device="cuda"), stream=Elsewhere())
    assert e.value.code == skv.SKV_ERR_ARG
