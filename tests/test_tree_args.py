"""Argument checks of the tree attention and the eviction (host side, no GPU)."""
import ctypes as C

import pytest
import torch

from long_context_decode_ada_b200 import skv


def size_of(ctx, B=2, N=8, Hq=8, Hkv=2, cap=100, positions=0, splits=7):
    n = C.c_size_t()
    rc = skv.lib().skv_tree_workspace_size(ctx.handle, B, N, Hq, Hkv, cap, positions, splits, C.byref(n))
    return rc, n.value


def test_workspace_grows_with_what_it_holds():
    ctx = skv.Context(16)
    base = size_of(ctx)
    assert base[0] == skv.SKV_OK and base[1] >= 2 * 7 * 8 * 4 * (128 * 4 + 8)
    for more in (dict(N=16), dict(Hkv=8, Hq=32, N=9), dict(splits=8), dict(positions=1), dict(splits=65535)):
        assert size_of(ctx, **more)[1] > base[1], more
    assert size_of(ctx, positions=1)[1] - base[1] >= 100 * 16 * 4


@pytest.mark.parametrize("bad", [dict(N=0), dict(N=65), dict(Hq=6), dict(Hq=7), dict(Hq=16), dict(Hkv=0),
                                 dict(B=-1), dict(cap=-1), dict(splits=-1), dict(splits=65536),
                                 dict(cap=1 << 26), dict(B=1 << 20)])
def test_sizes_outside_are_refused(bad):
    assert size_of(skv.Context(32), **bad)[0] == skv.SKV_ERR_ARG


def call(ctx, **kw):
    a = dict(q=0, qt=skv.Q_BF16, B=2, Hq=8, Hkv=2, N=4, K=0, V=0, kvt=skv.Q_FP16, qs=0, ks=0, cap=0.0,
             slopes=0, q_pos=0, splits=0)
    a.update(kw)
    t = skv.SkvTree(N=a["N"], kv_dtype=a["kvt"])
    t.K, t.V, t.q_stride, t.kv_stride = a["K"] or None, a["V"] or None, a["qs"], a["ks"]
    sc = skv.SkvScore(softcap=a["cap"])
    sc.slopes, sc.q_pos = a["slopes"] or None, a["q_pos"] or None
    pools = skv.SkvPools()
    return skv.lib().skv_tree_attention(
        ctx.handle, a["q"] or None, a["qt"], a["B"], a["Hq"], a["Hkv"], C.byref(t), C.byref(sc), None,
        None, None, 0, C.byref(pools), None, None, None, None, 0, a["splits"], None)


@pytest.mark.parametrize("bad", [
    dict(qt=7), dict(kvt=9), dict(K=16), dict(V=16), dict(qs=1000), dict(qs=1028), dict(ks=100),
    dict(ks=260), dict(cap=-1.0), dict(cap=float("inf")), dict(cap=float("nan")), dict(slopes=16),
    dict(N=0), dict(N=65), dict(Hq=24), dict(splits=-1), dict(splits=70000), dict()])
def test_calls_are_refused_before_the_gpu(bad):
    ctx = skv.Context(16)
    assert call(ctx, **bad) == skv.SKV_ERR_ARG                   # (the last: no buffers)
    assert len(skv.lib().skv_last_error()) > 10


@pytest.mark.parametrize("cap", [2.0 ** -41, 1e-45, 2.0 ** 41, 3e38])
def test_caps_outside_the_range_are_refused(cap):
    assert call(skv.Context(16), B=0, cap=cap) == skv.SKV_ERR_ARG
    assert call(skv.Context(16), B=0, cap=2.0 ** -40) == call(skv.Context(16), B=0, cap=2.0 ** 40) == skv.SKV_OK


def test_out_over_its_inputs_is_refused():
    for K, V, out in ((0, 0, 16), (32, 64, 32), (32, 64, 64)):
        t = skv.SkvTree(N=4, kv_dtype=skv.Q_FP16)
        t.K, t.V = K or None, V or None
        pools = skv.SkvPools()
        # (neither a workspace nor anything to read: the call cannot get past its checks)
        rc = skv.lib().skv_tree_attention(
            skv.Context(16).handle, 16, skv.Q_BF16, 2, 8, 2, C.byref(t), None, 128, None, None, 0,
            C.byref(pools), out, None, 128, None, 0, 0, None)
        assert rc == skv.SKV_ERR_ARG and b"out must not be" in skv.lib().skv_last_error()


def test_a_batch_of_none_and_bf16_stores():
    assert call(skv.Context(16), B=0) == skv.SKV_OK
    assert call(skv.Context(16, t0_bf16=True), B=0) == skv.SKV_ERR_ARG


def test_tree_masks():
    par = torch.tensor([[-1, 0, 0, 2], [-1, -1, 1, 2]])
    assert skv.tree_mask(par).tolist() == [[1, 3, 5, 13], [1, 2, 6, 14]]
    with pytest.raises(skv.SkvError):
        skv.tree_mask(torch.tensor([[-1, 2, 0]]))
    with pytest.raises(skv.SkvError):
        skv.tree_mask(torch.zeros((1, 65), dtype=torch.int64) - 1)


def test_evict_sizes():
    n = C.c_size_t()
    f = skv.lib().skv_evict_workspace_size
    ctx = skv.Context(64)
    assert f(ctx.handle, 2, 8, 1000, C.byref(n)) == skv.SKV_OK and n.value >= 4 * 16 * 1000
    for B, H, T in ((-1, 8, 10), (1, 0, 10), (1, 8, -1), (1, 8, (1 << 20) + 1), (1 << 20, 8, 10)):
        assert f(ctx.handle, B, H, T, C.byref(n)) == skv.SKV_ERR_ARG


def evict_call(indptr=16, ids=None, indptr_out=32, ids_out=None, cursor=48, cursor_out=None):
    """A store without tokens; no workspace: the call cannot get past its checks."""
    fl, pools = skv.SkvFreeLists(), skv.SkvPools()
    rc = skv.lib().skv_evict(
        skv.Context(16).handle, 1, 2, 0, 64, None, None, 80, 0, 0, None, None, indptr, ids, 0,
        C.byref(fl), cursor, C.byref(pools), None, None, indptr_out, None, ids_out, 0, cursor_out,
        96, None, 0, None)
    assert rc == skv.SKV_ERR_ARG
    return skv.lib().skv_last_error()


def test_evict_arrays_of_their_own():
    assert b"cursor" in evict_call(cursor_out=48)
    assert b"the old one's" in evict_call(indptr_out=16)
    assert b"the old one's" in evict_call(ids=128, ids_out=128)
    assert b"workspace" in evict_call(cursor_out=112)            # an empty store's NULLs are no overlap
