"""Eviction on the GPU: the kept set against a plain sort, tables and page
bytes exact, ties, held tokens, odd sizes, several blocks per unit, refusals,
and a run with the decode, the tree attention and the append around it."""
import ctypes as C

import numpy as np
import pytest
import torch

from long_context_decode_ada_b200 import skv
from long_context_decode_ada_b200 import workloads as wl
from _store64 import read_store, tree_reference
from test_gpu_tree import drafts

pytestmark = pytest.mark.gpu


def make_store(lens, Hkv=2, G=1, P=16, f=(0.2, 0.4, 0.3), seed=1, room=2, ctx_kw=None):
    quota = [[int(f[0] * T), int(f[1] * T), int(f[2] * T)] for T in lens]
    w = wl.custom(seed, len(lens), Hkv, G, P, lens, wl.MODE_QUOTA, quota=quota)
    w.pool_slots = [room * s + 2 for s in w.pool_slots]
    g = torch.Generator().manual_seed(seed)
    w.free_lists = [torch.randperm(s, generator=g).numpy().astype(np.uint32)
                    for s in w.pool_slots]
    ctx = skv.Context(P, **(ctx_kw or {}))
    dev = skv.workload_to_device(w)
    cache = skv.build_cache(ctx, w, dev)
    cache.check()
    return cache, dev


def kept_reference(tier, score, lens, keep, sink, recent, protect=None):
    """The tiers after the eviction, by a stable sort a unit."""
    out = np.full_like(tier, 3)
    B, H, Tmax = tier.shape
    for b in range(B):
        T = int(lens[b])
        for h in range(H):
            pos = [t for t in range(T) if tier[b, h, t] < 3]
            held = [t for t in pos if t < sink or t >= T - recent
                    or (protect is not None and protect[b, h, t])]
            rest = [t for t in pos if t not in set(held)]
            val = lambda t: -np.inf if np.isnan(score[b, h, t]) else score[b, h, t]  # noqa: E731
            # NaN behind everything, -inf included
            rest.sort(key=lambda t: (np.isnan(score[b, h, t]), -float(val(t)), t))
            more = max(0, int(keep[b]) - len(held))
            for t in held + rest[:more]:
                out[b, h, t] = tier[b, h, t]
    return out


def check_eviction(cache, new, want_tier, dev):
    """Tables in the allocation's layout, slots from the free lists, and every
    kept token's bytes as they were."""
    new.check()
    tier = new.tier.cpu().numpy()
    assert np.array_equal(tier, want_tier)
    B, H, Tmax = tier.shape
    P, U = cache.ctx.P, B * H
    row_of = new.row_of.cpu().numpy().reshape(U, Tmax)
    ptr = new.page_indptr.cpu().numpy()
    tip = new.page_tier_indptr.cpu().numpy()
    ids = new.page_ids.cpu().numpy().view(np.uint32)
    cur = cache.free_cursor().cpu().numpy()
    free = [f.cpu().numpy().view(np.uint32) for f in cache._free]
    at = 0
    took = [0, 0, 0]
    flat = tier.reshape(U, Tmax)
    for u in range(U):
        assert ptr[u] == at
        row = np.full(Tmax, -1)
        base = 0
        for t in range(3):
            assert tip[3 * u + t] == at
            pos = np.nonzero(flat[u] == t)[0]
            row[pos] = base + np.arange(len(pos))
            pages = -(-len(pos) // P)
            for k in range(pages):
                assert ids[at + k] == (t << 30) | int(free[t][cur[t] + took[t] + k])
            at += pages
            base += pages * P
            took[t] += pages
        assert np.array_equal(row_of[u], row)
    assert ptr[U] == at and tip[3 * U] == at
    assert np.array_equal(new.free_cursor().cpu().numpy(), cur + took)
    before, after = read_store(cache), read_store(new)
    for a, b, u in zip(before, after, range(U)):
        kept = np.nonzero(flat[u] < 3)[0]
        assert sorted(b["pos"].tolist()) == kept.tolist()
        old = {int(p): i for i, p in enumerate(a["pos"])}
        src = np.array([old[int(p)] for p in b["pos"]], dtype=np.int64)
        if len(src):
            assert np.array_equal(a["tier"][src], b["tier"])
            assert np.array_equal(a["K"][src], b["K"]) and np.array_equal(a["V"][src], b["V"])
    # headers name their unit and place; rows behind a page's last are zero
    pools = [p.cpu().numpy() for p in new.pools]
    for u in range(U):
        for k, g in enumerate(range(ptr[u], ptr[u + 1])):
            t, slot = int(ids[g]) >> 30, int(ids[g]) & 0x3FFFFFFF
            page = pools[t][slot * new.stride[t]: slot * new.stride[t] + new.payload[t]]
            first = int(tip[3 * u + t])
            assert page[4:16].view(np.uint32).tolist() == [u // H, u % H, g - first]
            n = int(page[0]) + 256 * int(page[1])
            if n < P:
                cb = (0, 64, 48)[t]
                if t == 0:
                    assert not page[16 + 256 * n:16 + 256 * P].any()
                else:
                    assert not page[16 + 2 * P + cb * n:16 + (2 + cb) * P].any()
                    assert not page[16 + 2 * n:16 + 2 * P].any()


def scores(shape, seed, zeros=0.1):
    g = torch.Generator().manual_seed(seed)
    s = torch.exp(2 * torch.randn(shape, generator=g))
    s[torch.rand(shape, generator=g) < zeros] = 0.0
    return s


CASES = [
    # lens, Hkv, P, keep, sink, recent
    ([300, 77], 2, 16, [100, 30], 4, 16),
    ([1], 1, 16, [1], 0, 0),
    ([1, 0, 5], 2, 16, [0, 3, 2], 0, 0),
    ([513, 64, 200], 2, 32, [40, 64, 1000], 0, 0),
    ([700, 129], 2, 64, [0, 10], 8, 8),
    ([257], 3, 64, [256], 300, 0),
    ([999, 1000], 1, 16, [-5, 500], 1, 1),
]


@pytest.mark.parametrize("lens,Hkv,P,keep,sink,recent", CASES)
def test_evict_against_a_sort(lens, Hkv, P, keep, sink, recent):
    cache, dev = make_store(lens, Hkv, 1, P, seed=sum(lens))
    shape = (len(lens), Hkv, max(lens))
    s = scores(shape, 3)
    new = cache.evict(s.cuda(), dev["seq_lens"], torch.tensor(keep, dtype=torch.int32).cuda(),
                      sink=sink, recent=recent)
    want = kept_reference(cache.tier.cpu().numpy(), s.numpy(), lens, keep, sink, recent)
    check_eviction(cache, new, want, dev)


@pytest.mark.parametrize("kind", ["zero", "ones", "nan", "mixed", "negative"])
def test_ties_and_unusual_scores(kind):
    lens = [400, 33]
    cache, dev = make_store(lens, 2, 1, 16, seed=5)
    s = scores((2, 2, 400), 9)
    if kind == "zero":
        s.zero_()
        s[:, :, ::3] = -0.0
    elif kind == "ones":
        s.fill_(1.0)
    elif kind == "nan":
        s.fill_(float("nan"))
    elif kind == "mixed":
        s[:, :, ::5] = float("nan")
        s[:, :, 1::5] = float("inf")
        s[:, :, 2::5] = -float("inf")
    else:
        s = -s
    keep = [150, 7]
    new = cache.evict(s.cuda(), dev["seq_lens"], torch.tensor(keep, dtype=torch.int32).cuda())
    want = kept_reference(cache.tier.cpu().numpy(), s.numpy(), lens, keep, 0, 0)
    check_eviction(cache, new, want, dev)


def test_protected_tokens_stay():
    lens = [300, 50]
    cache, dev = make_store(lens, 2, 1, 16, seed=6)
    s = scores((2, 2, 300), 4)
    g = torch.Generator().manual_seed(2)
    prot = (torch.rand((2, 2, 300), generator=g) < 0.2).to(torch.uint8)
    keep = [20, 40]
    new = cache.evict(s.cuda(), dev["seq_lens"], torch.tensor(keep, dtype=torch.int32).cuda(),
                      sink=2, recent=3, protect=prot.cuda())
    want = kept_reference(cache.tier.cpu().numpy(), s.numpy(), lens, keep, 2, 3, prot.numpy())
    check_eviction(cache, new, want, dev)


@pytest.mark.parametrize("kw", [dict(t1_angle_bits=5), dict(share_grid=1), dict(t0_bf16=True)])
def test_context_variants_move_bytes(kw):
    cache, dev = make_store([200], 2, 1, 16, seed=7, ctx_kw=kw)
    s = scores((1, 2, 200), 5)
    new = cache.evict(s.cuda(), dev["seq_lens"], torch.tensor([60], dtype=torch.int32).cuda())
    want = kept_reference(cache.tier.cpu().numpy(), s.numpy(), [200], [60], 0, 0)
    check_eviction(cache, new, want, dev)


@pytest.mark.parametrize("T", [16385, 40000, 140001])
def test_several_blocks_a_unit(T):
    cache, dev = make_store([T], 1, 1, 64, seed=8)
    s = scores((1, 1, T), 6, zeros=0.4)
    s = (s * 4).round() / 4                       # many equal scores across the blocks
    for keep in (T // 2, T // 3, 17):
        new = cache.evict(s.cuda(), dev["seq_lens"],
                          torch.tensor([keep], dtype=torch.int32).cuda(), sink=4, recent=64)
        new.check()
        tier = cache.tier.cpu()
        res = tier < 3
        pos = torch.arange(T)
        held = res & ((pos < 4) | (pos >= T - 64))
        more = max(0, keep - int(held.sum()))
        key = torch.where(res & ~held, s, torch.full_like(s, -1.0)).view(-1)
        order = torch.argsort(key, descending=True, stable=True)[:more]
        stay = held.view(-1).clone()
        stay[order[key[order] >= 0]] = True
        want = torch.where(stay.view_as(tier), tier, torch.full_like(tier, 3)).numpy()
        check_eviction(cache, new, want, dev)


@pytest.mark.parametrize("T", [4096, 4097, 8200, 32769, 65536, 131072, 131073])
def test_sizes_where_the_blocks_change(T):
    # 8 or 16 positions a thread, one to sixteen blocks a sequence's head, and the
    # first length beyond; sequences that end inside and rows off 16 bytes
    lens = [T, T // 3 + 1]
    cache, dev = make_store(lens, 1, 1, 64, f=(0.02, 0.3, 0.5), seed=T % 97)
    s = scores((2, 1, T), 3, zeros=0.3)
    s = (s * 8).round() / 8
    keep = torch.tensor([T // 2 + 3, 40], dtype=torch.int32)
    new = cache.evict(s.cuda(), dev["seq_lens"], keep.cuda(), sink=3, recent=33)
    new.check()
    tier = cache.tier.cpu()
    want = torch.full_like(tier, 3)
    pos = torch.arange(T)
    for b, L in enumerate(lens):
        res = (tier[b, 0] < 3) & (pos < L)
        held = res & ((pos < 3) | (pos >= L - 33))
        key = torch.where(res & ~held, s[b, 0], torch.full((T,), -1.0))
        order = torch.argsort(key, descending=True, stable=True)[:max(0, int(keep[b]) - int(held.sum()))]
        stay = held.clone()
        stay[order[key[order] >= 0]] = True
        want[b, 0] = torch.where(stay, tier[b, 0], want[b, 0])
    check_eviction(cache, new, want.numpy(), dev)


def test_long_store_without_cached_keys():
    # 2^20 positions: the scores are read again for every digit
    T = 1 << 20
    cache, dev = make_store([T], 1, 1, 64, f=(0.0, 0.0, 0.3), seed=9)
    s = scores((1, 1, T), 8, zeros=0.0)
    new = cache.evict(s.cuda(), dev["seq_lens"], torch.tensor([1000], dtype=torch.int32).cuda())
    new.check()
    tier = cache.tier.cpu().view(-1)
    key = torch.where(tier < 3, s.view(-1), torch.full((T,), -1.0))
    want = torch.full_like(tier, 3)
    top = torch.argsort(key, descending=True, stable=True)[:1000]
    want[top] = tier[top]
    assert torch.equal(new.tier.cpu().view(-1), want)


def test_pool_and_row_errors():
    cache, dev = make_store([300], 1, 1, 16, seed=10, room=1)
    s = scores((1, 1, 300), 2)
    keep = torch.tensor([290], dtype=torch.int32).cuda()
    before = [p.clone() for p in cache.pools]
    new = cache.evict(s.cuda(), dev["seq_lens"], keep)
    with pytest.raises(skv.SkvError) as e:
        new.check()
    assert e.value.code == skv.SKV_ERR_POOL
    n = int(cache.page_indptr[-1])
    for pid in cache.page_ids[:n].cpu().numpy().view(np.uint32):   # the old store is intact
        t, slot = int(pid) >> 30, int(pid) & 0x3FFFFFFF
        a, b = slot * cache.stride[t], (slot + 1) * cache.stride[t]
        assert torch.equal(cache.pools[t][a:b], before[t][a:b])
    cache, dev = make_store([300], 1, 1, 16, seed=10)
    first = int((cache.tier[0, 0] < 3).nonzero()[0])
    cache.row_of[0, 0, first] = 1 << 28
    new = cache.evict(s.cuda(), dev["seq_lens"], keep, sink=first + 1)
    with pytest.raises(skv.SkvError) as e:
        new.check()
    assert e.value.code == skv.SKV_ERR_CORRUPT


def test_a_store_without_tokens():
    ctx = skv.Context(16)
    fl, pools = skv.SkvFreeLists(), skv.SkvPools()
    i32 = lambda n, x: torch.full((n,), x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, keep, err, cursor, old = i32(2, 0), i32(2, 5), i32(1, 0), i32(3, 0), i32(7, 0)
    after, new, tiers = i32(3, -1), i32(7, -1), i32(19, -1)
    size = C.c_size_t()
    assert skv.lib().skv_evict_workspace_size(ctx.handle, 2, 3, 0, C.byref(size)) == skv.SKV_OK
    ws = torch.empty(max(size.value, 16), dtype=torch.uint8, device="cuda")
    at = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    rc = skv.lib().skv_evict(
        ctx.handle, 2, 3, 0, at(lens), None, None, at(keep), 1, 1, None, None, at(old), None, 0,
        C.byref(fl), at(cursor), C.byref(pools), None, None, at(new), at(tiers), None, 0, at(after),
        at(err), at(ws), ws.numel(), C.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == skv.SKV_OK, skv.lib().skv_last_error()
    torch.cuda.synchronize()
    assert new.eq(0).all() and tiers.eq(0).all() and int(err) == 0
    assert after.eq(0).all()


def test_refusals():
    cache, dev = make_store([100], 1, 1, 16, seed=11)
    s = scores((1, 1, 100), 2).cuda()
    keep = torch.tensor([50], dtype=torch.int32).cuda()
    for bad in (dict(score=s.double()), dict(score=s[..., :50]), dict(keep=keep.long()),
                dict(into=cache), dict(sink=-1), dict(recent=-1), dict(score=s.cpu())):
        kw = dict(score=s, seq_lens=dev["seq_lens"], keep=keep)
        kw.update(bad)
        with pytest.raises(skv.SkvError) as e:
            cache.evict(**kw)
        assert e.value.code == skv.SKV_ERR_ARG
    other, _ = make_store([100], 1, 1, 16, seed=12)
    with pytest.raises(skv.SkvError):
        cache.evict(s, dev["seq_lens"], keep, into=other.spare())


def test_captured_and_on_another_stream():
    cache, dev = make_store([700, 300], 2, 1, 16, seed=13)
    s = scores((2, 2, 700), 3).cuda()
    keep = torch.tensor([200, 100], dtype=torch.int32).cuda()
    into = cache.evict(s, dev["seq_lens"], keep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.evict(s, dev["seq_lens"], keep, into=into)
    s2 = scores((2, 2, 700), 30)
    s.copy_(s2)
    graph.replay()
    torch.cuda.synchronize()
    want = kept_reference(cache.tier.cpu().numpy(), s2.numpy(), [700, 300], [200, 100], 0, 0)
    check_eviction(cache, into, want, dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = cache.evict(s, dev["seq_lens"], keep)
    side.synchronize()
    check_eviction(cache, other, want, dev)


def test_a_serving_run():
    """Weights gathered by the decode, drafted tokens verified, the accepted
    ones appended, the store evicted, and the next tree verified on it."""
    lens = [600, 250]
    Hkv, G, N = 2, 4, 6
    quota = [[T // 5, T // 2, T // 4] for T in lens]
    w = wl.custom(14, 2, Hkv, G, 16, lens, wl.MODE_QUOTA, quota=quota)
    # room to grow
    Tmax = w.Tmax + 16
    ctx = skv.Context(16)
    dev = skv.workload_to_device(w)
    slots = [3 * x + 16 for x in w.pool_slots]
    cache = skv.PagedCache(ctx, 2, Hkv, Tmax, slots)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 16)).contiguous()  # noqa: E731
    K, V = pad(dev["K"]), pad(dev["V"])
    util = torch.nn.functional.pad(dev["utility"], (0, 16)).contiguous()
    free = [torch.randperm(s).to(torch.int32).cuda() for s in slots]
    seq = dev["seq_lens"].clone()
    cache.allocate(K, seq, util, None, wl.MODE_QUOTA, None, dev["quota"], free)
    cache.encode(K, V, seq)
    score = torch.zeros((2, Hkv, Tmax), device="cuda")
    for step in range(3):
        g = torch.Generator().manual_seed(step)
        qd = torch.randn((2, Hkv * G, 128), generator=g).to(torch.bfloat16).cuda()
        cache.decode_utility(qd.view(torch.int16), skv.Q_BF16, Hkv * G, seq, score)
    q, k, v, par = drafts(2, N, Hkv, G, 77)
    mask = skv.tree_mask(par).cuda()
    out, _ = cache.tree_attention(q, k, v, mask=mask)
    cache.check()
    o, _, ob, _ = tree_reference(cache, q, k=k, v=v, mask=mask.cpu())
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= ob)
    for j in (0, 1):                              # two tokens accepted
        cache.append(k[:, j].contiguous(), v[:, j].contiguous(), seq)
    cache.check()
    old_tier = cache.tier.cpu().numpy()
    keep = [200, 100]
    spare = cache.spare()
    new = cache.evict(score, seq, torch.tensor(keep, dtype=torch.int32).cuda(), sink=4, recent=16,
                      into=spare)
    want = kept_reference(old_tier, score.cpu().numpy(), seq.tolist(), keep, 4, 16)
    check_eviction(cache, new, want, dev)
    # the evicted store is a store: verified, appended to and decoded from
    out, _ = new.tree_attention(q, k, v, mask=mask)
    new.check()
    o, _, ob, _ = tree_reference(new, q, k=k, v=v, mask=mask.cpu())
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= ob)
    new.append(k[:, 2].contiguous(), v[:, 2].contiguous(), seq)
    new.check()
    a, _ = new.tree_attention(q[:, :1].contiguous())
    b, _ = new.decode(q[:, 0].contiguous().view(torch.int16), skv.Q_BF16, Hkv * G)
    new.check()
    tol = 2 * (1e-3 + 2e-3 * b.abs()) + 2.0 ** -8 * b.abs()
    assert torch.all((a[:, 0].float() - b).abs() <= tol)
