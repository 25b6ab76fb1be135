"""Tree attention over the paged store on the GPU against 64 bits: tiers, head
groups, page sizes, drafted tokens from one to 64, masks that leave rows
empty, ragged counts, capped and biased scores, strides, NaN and infinities in
masked places, bad pages, streams and graphs."""
import numpy as np
import pytest
import torch

from long_context_decode_ada_b200 import skv
from long_context_decode_ada_b200 import workloads as wl
from _store64 import tree_reference

pytestmark = pytest.mark.gpu


def make_store(lens, Hkv=2, G=4, P=16, f=(0.2, 0.4, 0.3), seed=1, slack=0, ctx_kw=None, **kw):
    quota = [[int(f[0] * T), int(f[1] * T), int(f[2] * T)] for T in lens]
    w = wl.custom(seed, len(lens), Hkv, G, P, lens, wl.MODE_QUOTA, quota=quota, scatter=True, **kw)
    ctx = skv.Context(P, **(ctx_kw or {}))
    dev = skv.workload_to_device(w)
    cache = skv.build_cache(ctx, w, dev)
    cache.check()
    return cache, dev


def drafts(B, N, Hkv, G, seed, qt=torch.bfloat16, kt=torch.float16):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, N, Hkv * G, 128), generator=g).to(qt).cuda()
    k = torch.randn((B, N, Hkv, 128), generator=g).to(kt).cuda()
    v = torch.randn((B, N, Hkv, 128), generator=g).to(kt).cuda()
    parents = torch.tensor([[-1] + [int(torch.randint(-1, i, (1,), generator=g)) for i in
                                    range(1, N)] for _ in range(B)])
    return q, k, v, parents


def compare(cache, got, q, **kw):
    out, lse = got
    cache.check()
    variant = {x: kw.pop(x) for x in ("t1_53", "lloyd") if x in kw}
    ref = {x: (y.cpu() if isinstance(y, torch.Tensor) else y) for x, y in kw.items()}
    o, l, ob, lb = tree_reference(cache, q, **ref, **variant)
    B, N = q.shape[:2]
    live = np.ones((B, N), bool)
    if kw.get("count") is not None:
        live = np.arange(N)[None] < kw["count"].cpu().numpy()[:, None]
    go = out.double().cpu().numpy()
    err = np.abs(go - o)
    assert np.all(err[live] <= ob[live]), \
        f"out: {int((err > ob)[live].sum())} of {ob[live].size}, worst {np.max((err / ob)[live]):.3g} of the bound"
    if lse is not None:
        gl = lse.double().cpu().numpy()
        fin = np.isfinite(l)
        assert np.array_equal(gl[live][~fin[live]], l[live][~fin[live]])
        e = np.abs(np.where(fin, gl, 0) - np.where(fin, l, 0))
        assert np.all(e[live] <= lb[live] + 1e-12), float(np.max((e / np.maximum(lb, 1e-12))[live]))
    return live


SHAPES = [
    # lens, Hkv, G, P, N
    ([300, 77], 2, 4, 16, 1),
    ([300, 77], 2, 4, 16, 5),
    ([1000, 1], 1, 1, 16, 3),
    ([513, 64, 0], 2, 2, 32, 8),
    ([700, 129], 2, 4, 64, 16),
    ([130, 65], 1, 4, 64, 33),
    ([900], 2, 4, 32, 64),
    ([1, 2, 3], 1, 2, 16, 64),
    ([2500], 8, 4, 64, 31),
]


@pytest.mark.parametrize("lens,Hkv,G,P,N", SHAPES)
@pytest.mark.parametrize("qt", [torch.bfloat16, torch.float16])
def test_tree_against_64_bits(lens, Hkv, G, P, N, qt):
    cache, _ = make_store(lens, Hkv, G, P, seed=len(lens) + N)
    B = len(lens)
    q, k, v, par = drafts(B, N, Hkv, G, 7 * N + P, qt, qt)
    mask = skv.tree_mask(par).cuda()
    lse = torch.full((B, N, Hkv * G), 7.0, device="cuda")
    got = cache.tree_attention(q, k, v, mask=mask, lse=lse)
    compare(cache, got, q, k=k, v=v, mask=mask)


@pytest.mark.parametrize("f", [(1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (0, 0, 0)])
@pytest.mark.parametrize("P", [16, 32, 64])
def test_single_tiers_and_nothing_resident(f, P):
    cache, _ = make_store([333, 40], 2, 2, P, f=f, seed=5)
    q, k, v, par = drafts(2, 6, 2, 2, 11)
    lse = torch.empty((2, 6, 4), device="cuda")
    compare(cache, cache.tree_attention(q, k, v, lse=lse), q, k=k, v=v)
    # the store alone
    out, lse = cache.tree_attention(q, lse=lse)
    compare(cache, (out, lse), q)
    if f == (0, 0, 0):
        assert torch.all(out == 0) and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("kw", [dict(ctx_kw=dict(t1_angle_bits=5)), dict(ctx_kw=dict(share_grid=1))])
def test_code_variants(kw):
    cache, _ = make_store([400, 90], 2, 4, 16, seed=3, **kw)
    q, k, v, par = drafts(2, 4, 2, 4, 1)
    v2 = dict(t1_53="t1_angle_bits" in kw["ctx_kw"], lloyd="share_grid" in kw["ctx_kw"])
    compare(cache, cache.tree_attention(q, k, v), q, k=k, v=v, **v2)


@pytest.mark.parametrize("kw", [dict(ctx_kw=dict(t1_angle_bits=5)), dict(ctx_kw=dict(share_grid=1))])
@pytest.mark.parametrize("N", [1, 12, 36])
def test_code_variants_at_other_row_counts(kw, N):
    cache, _ = make_store([260, 33], 2, 4, 32, seed=45, **kw)
    q, k, v, _ = drafts(2, N, 2, 4, 19)
    v2 = dict(t1_53="t1_angle_bits" in kw["ctx_kw"], lloyd="share_grid" in kw["ctx_kw"])
    compare(cache, cache.tree_attention(q, k, v), q, k=k, v=v, **v2)


@pytest.mark.parametrize("N", [2, 40])
def test_caps_that_some_scores_reach(N):
    # scores far above the cap beside small ones: both ways of the tanh
    cache, _ = make_store([1500], 1, 4, 64, seed=47, k_scale=4.0)
    q, k, v, _ = drafts(1, N, 1, 4, 23)
    q[:, :, 0] *= 8
    lse = torch.empty((1, N, 4), device="cuda")
    for cap in (2.0, 20.0, 500.0):
        got = cache.tree_attention(q, k, v, softcap=cap, lse=lse)
        compare(cache, got, q, k=k, v=v, softcap=cap)


@pytest.mark.parametrize("N", [1, 4, 40])
@pytest.mark.parametrize("cap", [1e4, 1e8, 2.0 ** 40])
def test_caps_far_above_the_scores(N, cap):
    cache, _ = make_store([700], 1, 4, 32, seed=53)
    q, k, v, _ = drafts(1, N, 1, 4, 29)
    lse = torch.empty((1, N, 4), device="cuda")
    compare(cache, cache.tree_attention(q, k, v, softcap=cap, lse=lse), q, k=k, v=v, softcap=cap)


@pytest.mark.parametrize("N", [2, 7, 40])
def test_a_row_beyond_the_cap_leaves_the_others(N):
    # the first token's scores pass a cap far above those of the others
    cache, _ = make_store([700], 1, 4, 32, seed=59)
    q, k, v, _ = drafts(1, N, 1, 4, 31)
    far = q.clone()
    far[:, 0] *= 2.0 ** 20
    lse, lse_far = (torch.empty((1, N, 4), device="cuda") for _ in range(2))
    got, _ = cache.tree_attention(q, k, v, softcap=1e5, lse=lse)
    got_far, _ = cache.tree_attention(far, k, v, softcap=1e5, lse=lse_far)
    assert torch.isfinite(got_far).all()
    got_far[:, 0], lse_far[:, 0] = got[:, 0], lse[:, 0]
    compare(cache, (got_far, lse_far), q, k=k, v=v, softcap=1e5)


@pytest.mark.parametrize("N,softcap,bias", [(1, 30.0, False), (7, 5.0, False), (1, 0.0, True),
                                            (20, 0.0, True), (33, 50.0, True)])
def test_capped_and_biased_scores(N, softcap, bias):
    lens = [612, 95, 0]
    cache, dev = make_store(lens, 2, 4, 32, seed=9, k_scale=3.0)
    q, k, v, par = drafts(3, N, 2, 4, 21)
    mask = skv.tree_mask(par).cuda()
    kw = dict(softcap=softcap)
    if bias:
        depth = torch.tensor([[bin(int(m) & (2 ** 64 - 1)).count("1") - 1 for m in row]
                              for row in mask.cpu()], dtype=torch.int32)
        kw["q_pos"] = (dev["seq_lens"].cpu()[:, None] + depth).to(torch.int32).cuda()
        kw["slopes"] = torch.tensor([2.0 ** -(i + 1) for i in range(8)], device="cuda")
    lse = torch.empty((3, N, 8), device="cuda")
    got = cache.tree_attention(q, k, v, mask=mask, lse=lse, seq_lens=dev["seq_lens"], **kw)
    compare(cache, got, q, k=k, v=v, mask=mask, **kw)


def test_large_scores_keep_their_order():
    # keys of three times the usual size and outliers: logits of tens to hundreds
    cache, _ = make_store([800], 2, 4, 16, seed=13, k_scale=12.0)
    q, k, v, par = drafts(1, 9, 2, 4, 2)
    lse = torch.empty((1, 9, 8), device="cuda")
    compare(cache, cache.tree_attention(q, k, v, lse=lse), q, k=k, v=v)
    big = (q.float() * 40).to(q.dtype)
    compare(cache, cache.tree_attention(big, k, v, lse=lse), big, k=k, v=v)


def test_ragged_counts_and_rows_left_as_they_were():
    lens = [500, 64, 31, 7]
    N = 12
    cache, _ = make_store(lens, 2, 4, 16, seed=4)
    q, k, v, par = drafts(4, N, 2, 4, 3)
    mask = skv.tree_mask(par).cuda()
    count = torch.tensor([12, 0, 5, 1], dtype=torch.int32, device="cuda")
    # what lies behind the counts is never read as a key, a value or a query
    for b, n in enumerate(count.tolist()):
        q[b, n:] = float("nan")
        k[b, n:] = float("inf")
        v[b, n:] = float("nan")
    out = torch.full_like(q, 3.0)
    lse = torch.full((4, N, 8), 5.0, device="cuda")
    got = cache.tree_attention(q, k, v, mask=mask, count=count, out=out, lse=lse)
    live = compare(cache, got, torch.nan_to_num(q), k=torch.nan_to_num(k, posinf=0.0),
                   v=torch.nan_to_num(v), mask=mask, count=count)
    dead = torch.from_numpy(~live)
    assert torch.all(out.cpu()[dead] == 3.0) and torch.all(lse.cpu()[dead] == 5.0)
    # counts outside 0..N are taken within it
    far = torch.tensor([99, -3, 5, 1], dtype=torch.int32, device="cuda")
    again, _ = cache.tree_attention(q, k, v, mask=mask, count=far, out=torch.full_like(q, 3.0))
    assert torch.equal(again, out)


def test_masks_that_leave_rows_empty():
    cache, _ = make_store([60, 0], 1, 4, 16, seed=6)
    q, k, v, _ = drafts(2, 5, 1, 4, 5)
    mask = torch.tensor([[0, 1, 2, 0, 31], [0, 1, 0, 4, 31]], dtype=torch.int64, device="cuda")
    lse = torch.empty((2, 5, 4), device="cuda")
    out, lse = cache.tree_attention(q, k, v, mask=mask, lse=lse)
    compare(cache, (out, lse), q, k=k, v=v, mask=mask)
    for i in (0, 2):
        assert torch.all(out[1, i] == 0) and torch.all(lse[1, i] == -float("inf"))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 65504.0])
def test_masked_places_may_hold_anything(bad):
    cache, _ = make_store([200], 2, 4, 16, seed=8)
    q, k, v, _ = drafts(1, 6, 2, 4, 9)
    mask = torch.tensor([[1, 3, 5, 9, 17, 33]], dtype=torch.int64, device="cuda")  # children of 0
    clean, _ = cache.tree_attention(q, k, v, mask=mask)
    k2, v2 = k.clone(), v.clone()
    k2[0, 2], v2[0, 2] = bad, bad
    got, _ = cache.tree_attention(q, k2, v2, mask=mask)
    cache.check()
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(got[:, keep], clean[:, keep])


def test_unused_rows_of_pages_may_hold_anything():
    cache, _ = make_store([77, 21], 2, 4, 64, seed=2)
    q, k, v, _ = drafts(2, 3, 2, 4, 4)
    clean, _ = cache.tree_attention(q, k, v)
    n = int(cache.page_indptr[-1])
    for pid in cache.page_ids[:n].cpu().numpy().view(np.uint32):
        page = cache.page_bytes_of(int(pid))
        head = page[:16].clone()
        rows, t = int(head[0]), int(pid) >> 30
        if rows == 64 or t == 0:
            continue
        cb = 64 if t == 1 else 48
        nan = torch.tensor([0x00, 0x7E], dtype=torch.uint8, device="cuda")  # fp16 NaN
        page[16 + 2 * rows:16 + 2 * 64] = nan.repeat(64 - rows)
        page[16 + (2 + cb) * 64 + 2 * rows:16 + (4 + cb) * 64] = nan.repeat(64 - rows)
    got, _ = cache.tree_attention(q, k, v)
    cache.check()
    assert torch.equal(got, clean)


def test_slices_of_a_fused_projection():
    B, N, Hkv, G = 2, 7, 2, 4
    cache, _ = make_store([150, 66], Hkv, G, 16, seed=15)
    g = torch.Generator().manual_seed(3)
    fused = torch.randn((B, N, (G + 2) * Hkv, 128), generator=g).to(torch.bfloat16).cuda()
    q, k, v = fused.split([G * Hkv, Hkv, Hkv], 2)
    assert not q.is_contiguous()
    out, _ = cache.tree_attention(q, k, v)
    want, _ = cache.tree_attention(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(out, want)
    compare(cache, (out, None), q, k=k, v=v)


@pytest.mark.parametrize("splits", [1, 2, 5, 37, 148, 600])
@pytest.mark.parametrize("by_bytes", [True, False])
def test_split_counts(splits, by_bytes):
    cache, _ = make_store([700, 0, 33, 410], 2, 4, 16, seed=17)
    cache.split_by_bytes = by_bytes
    q, k, v, par = drafts(4, 9, 2, 4, 8)
    mask = skv.tree_mask(par).cuda()
    lse = torch.empty((4, 9, 8), device="cuda")
    got = cache.tree_attention(q, k, v, mask=mask, lse=lse, num_splits=splits)
    compare(cache, got, q, k=k, v=v, mask=mask)


@pytest.mark.parametrize("N,n", [(17, 17), (20, 20), (24, 24), (40, 40), (16, 3), (40, 9)])
def test_rows_that_leave_lanes_idle(N, n):
    # long parts of a unit with rows for some of the warps only (68 to 96 rows of
    # 128, 160 of 256, or few rows of a batch that is laid out for many)
    cache, _ = make_store([9000, 2000], 1, 4, 16, seed=37, f=(0.05, 0.5, 0.4))
    q, k, v, par = drafts(2, N, 1, 4, N + n)
    mask = skv.tree_mask(par).cuda()
    count = torch.tensor([n, N], dtype=torch.int32, device="cuda")
    lse = torch.empty((2, N, 4), device="cuda")
    for splits in (3, 40):
        got = cache.tree_attention(q, k, v, mask=mask, count=count, lse=lse, num_splits=splits)
        again, _ = cache.tree_attention(q, k, v, mask=mask, count=count, num_splits=splits)
        cache.check()
        assert torch.equal(again[0, :n], got[0][0, :n]) and torch.equal(again[1], got[0][1])
    keep = [0, n - 1]
    one = dict(k=k[:, :n], v=v[:, :n], mask=mask[:, :n])
    ref = tree_reference(cache, q[:, :n].cpu(), **{a: b.cpu() for a, b in one.items()})
    out = got[0][0].double().cpu().numpy()
    for i in keep:
        err = np.abs(out[i] - ref[0][0, i])
        assert np.all(err <= ref[2][0, i]), float(np.max(err / ref[2][0, i]))


@pytest.mark.parametrize("N", [2, 5, 12, 33])
def test_long_runs(N):
    # one run with more pages of a unit than are held at once and more units than
    # are looked up at once, some of them empty or without drafted tokens
    lens = [9100] + [(37 * b) % 150 for b in range(21)]
    cache, _ = make_store(lens, 2, 4, 16, seed=49, f=(0.1, 0.5, 0.4))
    B = len(lens)
    q, k, v, _ = drafts(B, N, 2, 4, 27)
    count = torch.tensor([N if b % 4 != 2 else 0 for b in range(B)], dtype=torch.int32)
    lse = torch.empty((B, N, 8), device="cuda")
    outs = []
    for splits in (1, 3, 0):
        out, _ = cache.tree_attention(q, k, v, count=count.cuda(), lse=lse, num_splits=splits)
        outs.append(out)
    cache.check()
    # other runs round other sums: half a bf16 step and the weights' roundings apart
    for out in outs[:2]:
        assert torch.all((out.float() - outs[2].float()).abs() <= 2.0 ** -7 * outs[2].float().abs() + 4e-3)
    few = [0, 1, 2, 3, 21]
    sub = [x[few] for x in (q, k, v)]
    ref = tree_reference(_Part(cache, few), sub[0].cpu(), k=sub[1].cpu(), v=sub[2].cpu(), count=count[few])
    got = outs[0][few].double().cpu().numpy()
    for i, b in enumerate(few):
        n = int(count[b])
        assert np.all(np.abs(got[i, :n] - ref[0][i, :n]) <= ref[2][i, :n])
        assert torch.all(outs[0][b, n:] == 0)


class _Part:
    """Some sequences of a store, as tree_reference reads one."""

    def __init__(self, cache, seqs):
        self.ctx, self.Hkv, self.B = cache.ctx, cache.Hkv, len(seqs)
        self.pools, self.stride, self.payload = cache.pools, cache.stride, cache.payload
        ptr = cache.page_indptr.cpu()
        ids, to = [], [0]
        for b in seqs:
            for h in range(cache.Hkv):
                a, z = int(ptr[b * cache.Hkv + h]), int(ptr[b * cache.Hkv + h + 1])
                ids.append(cache.page_ids[a:z].cpu())
                to.append(to[-1] + z - a)
        self.page_indptr, self.page_ids = torch.tensor(to), torch.cat(ids)
        self.row_of = cache.row_of[seqs]


@pytest.mark.parametrize("N", [2, 6, 20, 40])      # 8, 24, 80 and 160 rows a kv head
def test_values_beyond_fp16(N):
    # drafted bf16 values that fp16 does not hold: the rows that see them get
    # them, the others the same bits as without
    cache, _ = make_store([700, 90], 2, 4, 16, seed=41)
    q, k, v, _ = drafts(2, N, 2, 4, 5, torch.bfloat16, torch.bfloat16)
    mask = torch.ones((2, N), dtype=torch.int64)
    mask[:, N - 1] = (1 << N) - 1                    # the last one sees all, the others token 0
    clean, _ = cache.tree_attention(q, k, v, mask=mask.cuda())
    v2 = v.clone()
    v2[0, 1, 0, 5], v2[0, 1, 1, 127], v2[1, N - 1, 1, 64] = 1e6, -3e5, 7e7
    lse = torch.empty((2, N, 8), device="cuda")
    got = cache.tree_attention(q, k, v2, mask=mask.cuda(), lse=lse)
    compare(cache, got, q, k=k, v=v2, mask=mask)
    assert torch.equal(got[0][:, :N - 1], clean[:, :N - 1])
    v2[0, 1, 0, 5], v2[0, 1, 0, 6] = float("inf"), float("nan")
    out = cache.tree_attention(q, k, v2, mask=mask.cuda())[0]
    assert torch.equal(out[:, :N - 1], clean[:, :N - 1])
    assert torch.all(out[0, N - 1, :4, 5] == float("inf")) and torch.isnan(out[0, N - 1, :4, 6]).all()


@pytest.mark.parametrize("N", [2, 6, 20, 40])
def test_a_query_that_is_not_a_number_stays_in_its_row(N):
    cache, _ = make_store([900], 2, 4, 32, seed=43)
    q, k, v, _ = drafts(1, N, 2, 4, 15)
    clean, _ = cache.tree_attention(q, k, v)
    q[0, 1, 3] = float("nan")
    lse = torch.empty((1, N, 8), device="cuda")
    out, _ = cache.tree_attention(q, k, v, lse=lse)
    assert torch.isnan(out[0, 1, 3]).all() and torch.isnan(lse[0, 1, 3])
    out[0, 1, 3] = clean[0, 1, 3]
    assert torch.equal(out, clean)


def test_same_result_every_call_and_after_other_sizes():
    cache, _ = make_store([3000, 900], 2, 4, 64, seed=19)
    q, k, v, par = drafts(2, 24, 2, 4, 6)
    first, _ = cache.tree_attention(q, k, v)
    ws = cache.tree_workspace(64, 8)
    ws.fill_(0xFF)                                  # the workspace needs no initialisation
    for n in (1, 64, 24):
        cache.tree_attention(*[x[:, :1].repeat(1, n, 1, 1) for x in (q, k, v)], workspace=ws)
        again, _ = cache.tree_attention(q, k, v, workspace=ws)
        assert torch.equal(again, first)
    cache.check()


def test_streams_and_graphs():
    cache, _ = make_store([1200, 50], 2, 4, 32, seed=23)
    q, k, v, par = drafts(2, 10, 2, 4, 12)
    mask = skv.tree_mask(par).cuda()
    want, _ = cache.tree_attention(q, k, v, mask=mask)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [torch.zeros_like(q) for _ in range(2)]
    wss = [cache.tree_workspace(10, 8) for _ in range(2)]
    with torch.cuda.stream(side):
        cache.tree_attention(q, k, v, mask=mask, out=outs[0], workspace=wss[0])
    cache.tree_attention(q, k, v, mask=mask, out=outs[1], workspace=wss[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # a captured call follows its inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.tree_attention(q, k, v, mask=mask, out=outs[0], workspace=wss[0])
    other = torch.randn_like(q.float()).to(q.dtype)
    q.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    want, _ = cache.tree_attention(q, k, v, mask=mask)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    cache.check()


def test_bad_pages_and_rows_are_reported():
    cache, dev = make_store([300], 1, 4, 16, seed=27)
    q, k, v, _ = drafts(1, 4, 1, 4, 14)
    good = cache.page_ids.clone()
    for wrong in (0x3FFFFFFF, (3 << 30) - (1 << 32), (1 << 30) | 0x3FFFFFF):
        cache.page_ids.copy_(good)
        cache.page_ids[3] = wrong
        cache.tree_attention(q, k, v)
        with pytest.raises(skv.SkvError) as e:
            cache.check()
        assert e.value.code == skv.SKV_ERR_CORRUPT
    cache.page_ids.copy_(good)
    row = cache.row_of.clone()
    cache.row_of[0, 0, 5] = 1 << 29
    slopes = torch.zeros(4, device="cuda")
    q_pos = torch.full((1, 4), 300, dtype=torch.int32, device="cuda")
    cache.tree_attention(q, k, v, slopes=slopes, q_pos=q_pos, seq_lens=dev["seq_lens"])
    with pytest.raises(skv.SkvError) as e:
        cache.check()
    assert e.value.code == skv.SKV_ERR_CORRUPT
    cache.row_of.copy_(row)
    out, _ = cache.tree_attention(q, k, v)
    compare(cache, (out, None), q, k=k, v=v)


def test_agrees_with_the_single_token_decode():
    cache, dev = make_store([2000, 300], 2, 4, 64, seed=31)
    q = dev["q"].view(torch.bfloat16).view(2, 1, 8, 128)
    ref, rl = cache.decode(dev["q"], dev["q_dtype"], 8)
    lse = torch.empty((2, 1, 8), device="cuda")
    out, _ = cache.tree_attention(q, lse=lse)
    cache.check()
    # both within the decode's bound of the exact value, and out once rounded to bf16
    tol = 2 * (1e-3 + 2e-3 * ref.abs()) + 2.0 ** -8 * ref.abs()
    assert torch.all((out.float().view_as(ref) - ref).abs() <= tol)
    assert torch.all((lse.view_as(rl) - rl).abs() <= 2 * (1e-3 + 2e-3 * rl.abs()))
