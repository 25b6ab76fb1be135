"""Measured cases of the operators that verify drafted tokens over the paged
store and evict from it.

Two operators:

- ``verify``: attention of N drafted tokens a sequence (a tree: every token
  sees the store and its own ancestors) over the paged store of dense (T0)
  and coded (T1, T2) keys and values, the scores optionally capped by a tanh
  or biased by distance; N = 1 without drafted keys is the single-token form.
- ``evict``: the store without the tokens of least accumulated attention
  weight: per (sequence, kv head) the sink, the recent window and the highest
  scores stay, in their tier and with their bytes, in newly packed pages.

``run`` computes a pass in plain torch operations, or, where ``own`` is true,
by the calls a user makes.  The store is made by ``prepare`` from seeded keys
and values (header 16 B; T0: fp16 K and V; T1: radius, 6-bit angle and 2-bit
share a pair, int8 V with a scale; T2: the same with a 4-bit angle).
"""
import math

import numpy as np
import torch

own = False

D = 128                                   # head size
PAIRS = 64
ROW_BYTES = (512, 196, 180)               # a token of each tier
DROP = 3


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a small all-T2 store of one head, a chain of four drafted tokens
        dict(name="verify_tiny", op="verify", B=1, Hkv=1, G=1, P=16, Tlo=4096, T=4096,
             f0=0.0, f1=0.0, f2=1.0, N=4, draft=True, chain=True, ragged=False, cap=0.0,
             bias=False, q="fp16"),
        # one conversation of some thousand tokens, a tree of eight
        dict(name="verify_chat", op="verify", B=1, Hkv=8, G=4, P=64, Tlo=5003, T=5003,
             f0=0.1, f1=0.5, f2=0.25, N=8, draft=True, chain=False, ragged=False, cap=0.0,
             bias=False, q="bf16"),
        # the serving batch: ragged lengths, scattered pages, trees of up to eight
        dict(name="verify_ragged", op="verify", B=64, Hkv=8, G=4, P=16, Tlo=1024, T=8192,
             f0=0.2, f1=0.4, f2=0.4, N=8, draft=True, chain=False, ragged=True, cap=0.0,
             bias=False, q="bf16"),
        # a batch of long prompts, chains of sixteen
        dict(name="verify_layer", op="verify", B=8, Hkv=8, G=4, P=64, Tlo=32768, T=32768,
             f0=0.1, f1=0.5, f2=0.25, N=16, draft=True, chain=True, ragged=False, cap=0.0,
             bias=False, q="bf16"),
        # the 128K context under its budget, trees of 32 and 64 (the largest)
        dict(name="verify_128k_32", op="verify", B=1, Hkv=8, G=4, P=64, Tlo=131072, T=131072,
             f0=0.01, f1=0.99, f2=0.0, N=32, draft=True, chain=False, ragged=False, cap=0.0,
             bias=False, q="bf16"),
        dict(name="verify_128k_64_capped", op="verify", B=1, Hkv=8, G=4, P=64, Tlo=131072,
             T=131072, f0=0.01, f1=0.99, f2=0.0, N=64, draft=True, chain=False, ragged=False,
             cap=30.0, bias=False, q="bf16"),
        # one new token a sequence: capped over the 128K context, biased by
        # distance over the serving batch
        dict(name="token_128k_capped", op="verify", B=1, Hkv=8, G=4, P=64, Tlo=131072, T=131072,
             f0=0.01, f1=0.99, f2=0.0, N=1, draft=False, chain=True, ragged=False, cap=50.0,
             bias=False, q="bf16"),
        dict(name="token_ragged_biased", op="verify", B=64, Hkv=8, G=4, P=16, Tlo=1024, T=8192,
             f0=0.2, f1=0.4, f2=0.4, N=1, draft=False, chain=True, ragged=False, cap=0.0,
             bias=True, q="bf16"),
        # half of a small one-head store
        dict(name="evict_tiny", op="evict", B=1, Hkv=1, P=16, Tlo=4096, T=4096, f0=0.0, f1=0.0,
             f2=1.0, keep=2048, sink=4, recent=64),
        # the serving batch brought down to 2048 tokens a head
        dict(name="evict_ragged", op="evict", B=64, Hkv=8, P=16, Tlo=1024, T=8192, f0=0.2,
             f1=0.4, f2=0.4, keep=2048, sink=16, recent=256),
        # a batch of long prompts to a quarter
        dict(name="evict_layer", op="evict", B=8, Hkv=8, P=64, Tlo=32768, T=32768, f0=0.1,
             f1=0.5, f2=0.25, keep=8192, sink=64, recent=1024),
        # the 128K context to half
        dict(name="evict_128k", op="evict", B=1, Hkv=8, P=64, Tlo=131072, T=131072, f0=0.01,
             f1=0.99, f2=0.0, keep=65536, sink=64, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    B = _log(rng, 1, 64)
    Hkv = rng.choice([1, 2, 4, 8])
    P = rng.choice([16, 32, 64])
    T = _log(rng, 16, max(16, min(131072, 2_000_000 // (B * Hkv))))
    f0 = round(rng.uniform(0.0, 0.25), 3)
    f1 = round(rng.uniform(0.0, 1.0 - f0), 3)
    f2 = round(rng.uniform(0.0, 1.0 - f0 - f1), 3)
    c = dict(op=rng.choice(["verify", "verify", "evict"]), B=B, Hkv=Hkv, P=P,
             Tlo=rng.randint(1, T), T=T, f0=f0, f1=f1, f2=f2)
    if c["op"] == "evict":
        c.update(keep=rng.randint(1, T), sink=rng.choice([0, 4, 16, 64]),
                 recent=rng.choice([0, 1, 64, 256, 1024]))
        return c
    G = rng.choice([1, 2, 4])
    rows = max(1, B * Hkv * T)
    # at most the products of 64 tokens of four heads over the 128K context
    c.update(G=G, N=min(_log(rng, 1, 64), max(1, 256 * 8 * 131072 // (rows * G))),
             draft=rng.random() < 0.8, chain=rng.random() < 0.4, ragged=rng.random() < 0.4,
             cap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.3,
             q=rng.choice(["bf16", "bf16", "fp16"]))
    return c


def _lens(c):
    """Lengths of the sequences, spread over [Tlo, T] (known without a seed)."""
    B = c["B"]
    if B == 1:
        return [c["T"]]
    step = 7 if B % 7 else 11
    return [c["Tlo"] + (c["T"] - c["Tlo"]) * ((b * step) % B) // (B - 1) for b in range(B)]


def _tiers(c, T):
    n0, n1 = int(c["f0"] * T), int(c["f1"] * T)
    return n0, n1, min(T - n0 - n1, int(c["f2"] * T + 0.5))


def _counts(c):
    """Drafted tokens of each sequence: N, or ragged from none to N."""
    N, B = c["N"], c["B"]
    return [N if not c["ragged"] else (N * ((b + 3) % 4) + 2) // 3 for b in range(B)]


def work(c):
    lens = _lens(c)
    n = [_tiers(c, T) for T in lens]
    if c["op"] == "evict":
        # the score, tier and row of every position, and the new tier and row;
        # a kept row read and written (the kept rows' tiers in proportion)
        total = 0.0
        for T, t in zip(lens, n):
            have = max(1, sum(t))
            kept = min(c["keep"], have)
            total += T * (4 + 1 + 4 + 1 + 4)
            total += 2.0 * kept * sum(x * b for x, b in zip(t, ROW_BYTES)) / have
        return {"bytes": total * c["Hkv"], "flops": 0}
    G, Hkv, N = c["G"], c["Hkv"], c["N"]
    nbytes, flops = 0.0, 0.0
    for T, t, m in zip(lens, n, _counts(c)):
        if m == 0:
            continue
        nbytes += Hkv * sum(x * b for x, b in zip(t, ROW_BYTES))
        nbytes += m * Hkv * (2 * G * D * 2 + (2 * D * 2 if c["draft"] else 0))
        nbytes += 4 * Hkv * T if c["bias"] else 0
        flops += 4.0 * D * Hkv * G * m * (sum(t) + (m if c["draft"] else 0))
    return {"bytes": max(nbytes, 1.0), "flops": flops}


# ------------------------------------------------------- the store's layout
def _page_bytes(t, P):
    pay = 16 + P * ROW_BYTES[t]
    return pay, (pay + 127) // 128 * 128


def _v_index(P):
    """[P][128] element index of (row, dim) in a page's V section (blocks of 8
    rows; dims and rows interleaved in matrix-fragment order), by element size."""
    r = torch.arange(P).view(P, 1)
    d = torch.arange(D).view(1, D)
    k, t4, lo = r // 8, r % 8 // 2, r % 2
    mt, g, hi = d // 16, d % 8, d % 16 // 8
    L, e = 4 * g + t4, 2 * hi + lo
    one = k * 1024 + 512 * (mt // 4) + 16 * L + 4 * (mt % 4) + e
    two = k * 1024 + 256 * (mt // 2) + 8 * L + 4 * (mt % 2) + e
    return one, two


def _pair_place():
    """Per pair: its lane group g (of four) and its place j in the group."""
    p = torch.arange(PAIRS)
    return p % 16 // 4, 4 * (p // 16) + p % 4


def _layout(P, device):
    one, two = _v_index(P)
    g, j = _pair_place()
    r = torch.arange(P).view(P, 1)
    d = torch.arange(D).view(1, D)
    k0 = 128 * r + 8 * ((d // 8) ^ (4 * (r % 2))) + d % 8
    put = lambda x: x.to(device)  # noqa: E731
    return dict(v1=put(one.reshape(-1)), v2=put(two.reshape(-1)), k0=put(k0.reshape(-1)),
                code1=put(16 * g + j), angle2=put(8 * g + j // 2), odd2=put(j % 2),
                share2=put(32 + 4 * g + j // 4), bits2=put(2 * (j % 4)))


def _pack_rows(t, P, lay, K, V):
    """Pages [n][payload - 16] of n x P rows of fp16 keys and values."""
    n = K.shape[0] // P
    if t == 0:
        body = torch.empty((n, 2 * P * D), dtype=torch.float16, device=K.device)
        body[:, lay["k0"]] = K.view(n, P * D)
        body[:, P * D + lay["v2"]] = V.view(n, P * D)
        return body.view(torch.uint8)
    Kf, Vf = K.float(), V.float()
    r = Kf.square().sum(1).sqrt()
    x, y = Kf[:, 0::2], Kf[:, 1::2]
    bits = 6 if t == 1 else 4
    a = torch.round(torch.atan2(y, x) * ((1 << bits) / (2 * math.pi))).to(torch.int32) % (1 << bits)
    u = (x * x + y * y).sqrt() * 8.0 / r.clamp_min(1e-30).unsqueeze(1)
    s = (u > 0.75).to(torch.int32) + (u > 1.25) + (u > 1.75)
    cb = 64 if t == 1 else 48
    codes = torch.zeros((n * P, cb), dtype=torch.int32, device=K.device)
    if t == 1:
        codes[:, lay["code1"]] = 4 * a + s
    else:
        codes.index_add_(1, lay["angle2"], a << (4 * lay["odd2"]).to(torch.int32))
        codes.index_add_(1, lay["share2"], s << lay["bits2"].to(torch.int32))
    sc = (Vf.abs().amax(1) / 127.0).to(torch.float16)
    v8 = torch.round(Vf / sc.float().clamp_min(1e-30).unsqueeze(1)).clamp(-127, 127).to(torch.int8)
    body = torch.empty((n, P * ROW_BYTES[t]), dtype=torch.uint8, device=K.device)
    body[:, :2 * P] = r.to(torch.float16).view(n, P).view(torch.uint8)
    body[:, 2 * P:(2 + cb) * P] = codes.to(torch.uint8).view(n, P * cb)
    body[:, (2 + cb) * P:(4 + cb) * P] = sc.view(n, P).view(torch.uint8)
    vsec = torch.empty((n, P * D), dtype=torch.uint8, device=K.device)
    vsec[:, lay["v1"]] = v8.view(n, P * D).view(torch.uint8)
    body[:, (4 + cb) * P:] = vsec
    return body


def _tables(tier, P, B, Hkv):
    """Row map and page table of a tier array: (row_of, tier_indptr, pages per
    (unit, tier))."""
    U = B * Hkv
    flat = tier.view(U, -1)
    row_of = torch.full_like(flat, -1, dtype=torch.int32)
    n, idx = [], []
    for t in range(3):
        hit = flat == t
        idx.append((hit, torch.cumsum(hit, 1, dtype=torch.int32) - 1))
        n.append(hit.sum(1))
    pages = torch.stack([(x + P - 1) // P for x in n], 1)           # [U][3]
    first = torch.cumsum(pages, 1) - pages                          # within the unit
    for t in range(3):
        hit, i = idx[t]
        row_of = torch.where(hit, i + (first[:, t:t + 1] * P).to(torch.int32), row_of)
    tip = torch.zeros(3 * U + 1, dtype=torch.int32, device=tier.device)
    tip[1:] = torch.cumsum(pages.view(-1), 0)
    return row_of.view(tier.shape), tip, pages, torch.stack(n, 1)


def _page_ids(pages, free, cursor):
    """Page ids in list order: per (unit, tier) segment, slots in unit order."""
    U = pages.shape[0]
    seg = torch.repeat_interleave(torch.arange(3 * U, device=pages.device), pages.view(-1))
    ids = torch.zeros(seg.numel(), dtype=torch.int64, device=pages.device)
    for t in range(3):
        mine = seg % 3 == t
        k = torch.cumsum(mine, 0)[mine] - 1
        ids[mine] = free[t][k + cursor[t]].to(torch.int64) | (t << 30)
    return ids, seg


def _headers(ids, seg, n, P, Hkv, tip):
    """The 16-byte headers of the listed pages, as int32 words."""
    u, t = seg // 3, seg % 3
    inseg = torch.arange(seg.numel(), device=seg.device) - tip[seg].long()
    rows = (n.view(-1)[seg] - inseg * P).clamp(max=P)
    w = torch.stack([rows | (t << 16) | (0x5A << 24), u // Hkv, u % Hkv, inseg], 1)
    return w.to(torch.int32)


def _make_store(c, gen, dev, spare):
    """A paged store of seeded keys and values, with `spare` free slots a tier
    beyond the pages in use; every tensor that a user's program holds of it."""
    B, Hkv, P, lens = c["B"], c["Hkv"], c["P"], _lens(c)
    Tmax = max(max(lens), 1)
    U = B * Hkv
    L = torch.tensor(lens, dtype=torch.int32, device=dev)
    pos = torch.arange(Tmax, device=dev)
    live = pos.view(1, 1, -1) < L.view(B, 1, 1)
    u = torch.rand((B, Hkv, Tmax), generator=gen, device=dev)
    u = torch.where(live, u, torch.full_like(u, 2.0))
    rank = torch.empty((B, Hkv, Tmax), dtype=torch.int32, device=dev)
    rank.scatter_(2, u.argsort(2), pos.to(torch.int32).expand(B, Hkv, Tmax).contiguous())
    quota = torch.tensor([_tiers(c, T) for T in lens], dtype=torch.int32, device=dev)
    edge = torch.cumsum(quota, 1).view(B, 1, 1, 3)
    tier = (rank.unsqueeze(-1) >= edge).sum(-1).to(torch.uint8)
    tier = torch.where(live, tier, torch.full_like(tier, DROP))
    row_of, tip, pages, n = _tables(tier, P, B, Hkv)
    used = [int(x) for x in pages.sum(0)]
    slots = [used[t] + spare(t, used[t]) for t in range(3)]
    free = [torch.randperm(max(slots[t], 1), generator=gen, device=dev)[:slots[t]].to(torch.int32)
            for t in range(3)]
    cursor = torch.tensor(used, dtype=torch.int32, device=dev)
    ids, seg = _page_ids(pages, free, [0, 0, 0])
    hdr = _headers(ids, seg, n, P, Hkv, tip)
    lay = _layout(P, dev)
    scale = torch.exp(0.5 * torch.randn((U, D), generator=gen, device=dev))
    pools = []
    for t in range(3):
        pay, stride = _page_bytes(t, P)
        pool = torch.zeros((max(slots[t], 1), stride), dtype=torch.uint8, device=dev)
        mine = seg % 3 == t
        np_t = int(mine.sum())
        if np_t:
            slot = ids[mine] & 0x3FFFFFFF
            unit = seg[mine] // 3
            K = torch.randn((np_t, P, D), generator=gen, device=dev) * scale[unit].unsqueeze(1)
            V = torch.randn((np_t, P, D), generator=gen, device=dev)
            rows = (hdr[mine, 0] & 0xFFFF).view(-1, 1, 1)
            gone = torch.arange(P, device=dev).view(1, P, 1) >= rows
            K = K.masked_fill_(gone, 0.0).to(torch.float16).view(-1, D)
            V = V.masked_fill_(gone, 0.0).to(torch.float16).view(-1, D)
            page = torch.zeros((np_t, stride), dtype=torch.uint8, device=dev)
            page[:, :16] = hdr[mine].contiguous().view(torch.uint8).view(-1, 16)
            page[:, 16:pay] = _pack_rows(t, P, lay, K, V)
            pool[slot] = page
        pools.append(pool)
    cap = int(pages.sum())
    page_ids = ids.to(torch.int32)
    return dict(c=c, B=B, Hkv=Hkv, P=P, Tmax=Tmax, seq_lens=L, tier=tier, row_of=row_of,
                tip=tip, indptr=tip[0::3].contiguous(), page_ids=page_ids, cap=cap, pools=pools,
                slots=slots, free=free, cursor=cursor, lay=lay)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1_000_003 * (int(seed) + 1) + len(str(case)))
    c = dict(case)
    if c["op"] == "evict":
        # room for the packed pages beside the old ones
        st = _make_store(c, gen, dev, lambda t, n: n)
        shape = (st["B"], st["Hkv"], st["Tmax"])
        # accumulated weights: heavy-tailed, some tokens never looked at
        score = torch.exp(2.0 * torch.randn(shape, generator=gen, device=dev))
        score.masked_fill_(torch.rand(shape, generator=gen, device=dev) < 0.05, 0.0)
        st.update(score=score, keep=torch.full((st["B"],), c["keep"], dtype=torch.int32,
                                               device=dev))
        if own:
            st["cache"] = _cache(st)
            st["into"] = st["cache"].spare()
        else:
            st["new"] = dict(ids=torch.zeros(max(1, st["cap"]), dtype=torch.int32, device=dev))
        return st
    st = _make_store(c, gen, dev, lambda t, n: 0)
    B, N, Hkv, G = c["B"], c["N"], c["Hkv"], c["G"]
    qt = torch.bfloat16 if c["q"] == "bf16" else torch.float16
    st["q"] = torch.randn((B, N, Hkv * G, D), generator=gen, device=dev).to(qt)
    st["out"] = torch.zeros((B, N, Hkv * G, D), dtype=qt, device=dev)
    st["k"] = st["v"] = st["mask"] = st["q_pos"] = st["slopes"] = None
    st["count"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev)
    # a tree: token i hangs under an earlier token (the chain: under the last)
    depth = torch.zeros((B, N), dtype=torch.int32, device=dev)
    bits = torch.zeros((B, N), dtype=torch.int64, device=dev)
    pick = torch.rand((B, N), generator=gen, device=dev)
    for i in range(N):
        par = torch.full((B,), i - 1, dtype=torch.int64, device=dev) if c["chain"] else \
            (pick[:, i] * (i + 1)).long().clamp(max=i) - 1
        up = par.clamp(min=0).view(B, 1)
        has = (par >= 0).view(B, 1)
        one = -(1 << 63) if i == 63 else 1 << i
        bits[:, i] = (bits.gather(1, up) * has).view(B) | one
        depth[:, i] = (torch.where(has, depth.gather(1, up) + 1, torch.zeros_like(up))).view(B)
    if c["draft"]:
        st["k"] = torch.randn((B, N, Hkv, D), generator=gen, device=dev).to(torch.float16)
        st["v"] = torch.randn((B, N, Hkv, D), generator=gen, device=dev).to(torch.float16)
        st["mask"] = bits
    if c["bias"]:
        Hq = Hkv * G
        st["q_pos"] = st["seq_lens"].view(B, 1) + depth
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)],
                                    dtype=torch.float32, device=dev)
    if own:
        st["cache"] = _cache(st)
        st["ws"] = st["cache"].tree_workspace(N, Hkv * G, positions=c["bias"])
    return st


def _cache(st):
    """The prepared store as the framework's paged cache."""
    from long_context_decode_ada_b200 import skv
    cache = skv.PagedCache(skv.Context(st["P"]), st["B"], st["Hkv"], st["Tmax"], st["slots"],
                           page_cap=st["cap"])
    for t in range(3):
        cache.pools[t].copy_(st["pools"][t].view(-1))
    cache.tier.copy_(st["tier"])
    cache.row_of.copy_(st["row_of"])
    cache.page_indptr.copy_(st["indptr"])
    cache.page_tier_indptr.copy_(st["tip"])
    if st["cap"]:
        cache.page_ids.copy_(st["page_ids"])
    cache.set_free_lists(st["free"], st["cursor"])
    st["pools"] = None
    return cache


def run(state):
    if own:
        cache, c = state["cache"], state["c"]
        if c["op"] == "evict":
            new = cache.evict(state["score"], state["seq_lens"], state["keep"], sink=c["sink"],
                              recent=c["recent"], into=state["into"])
            return dict(tier=new.tier, row_of=new.row_of, indptr=new.page_indptr,
                        tier_indptr=new.page_tier_indptr, page_ids=new.page_ids,
                        pools=[p.view(max(1, s), -1) for p, s in zip(new.pools, new.pool_slots)])
        out, _ = cache.tree_attention(state["q"], state["k"], state["v"], mask=state["mask"],
                                      count=state["count"], softcap=c["cap"],
                                      slopes=state["slopes"], q_pos=state["q_pos"],
                                      seq_lens=state["seq_lens"], out=state["out"],
                                      workspace=state["ws"])
        return out
    return _evict(state) if state["c"]["op"] == "evict" else _verify(state)


# -------------------------------------------------------------- plain forms
def _rows(t, P, lay, page):
    """fp32 keys and values [n][P][128] of pages [n][stride] of tier t."""
    n = page.shape[0]
    pay = 16 + P * ROW_BYTES[t]
    if t == 0:
        h = page[:, 16:pay].contiguous().view(torch.float16)
        return (h[:, lay["k0"]].view(n, P, D).float(),
                h[:, P * D + lay["v2"]].view(n, P, D).float())
    cb = 64 if t == 1 else 48
    half = lambda at: page[:, at:at + 2 * P].contiguous().view(torch.float16).float()  # noqa: E731
    r, sc = half(16), half(16 + (2 + cb) * P)
    codes = page[:, 16 + 2 * P:16 + (2 + cb) * P].reshape(n, P, cb)
    if t == 1:
        w = codes[:, :, lay["code1"]].int()
        a, s, step = w >> 2, w & 3, 2 * math.pi / 64
    else:
        a = (codes[:, :, lay["angle2"]].int() >> (4 * lay["odd2"])) & 15
        s = (codes[:, :, lay["share2"]].int() >> lay["bits2"]) & 3
        step = 2 * math.pi / 16
    # the angles from 64 bits, rounded once
    th = torch.arange(64, device=page.device, dtype=torch.float64) * step
    mag = (s + 1).float() * (r / 16.0).unsqueeze(-1)
    K = torch.stack([mag * th.cos().float()[a.long()], mag * th.sin().float()[a.long()]], -1)
    v = page[:, 16 + (4 + cb) * P:pay][:, lay["v1"]].contiguous().view(torch.int8)
    return K.view(n, P, D), v.view(n, P, D).float() * sc.unsqueeze(-1)


def _verify(st):
    c, P, B, Hkv = st["c"], st["P"], st["B"], st["Hkv"]
    N, G, U, dev = c["N"], c["G"], st["B"] * st["Hkv"], st["q"].device
    Hq, R = Hkv * G, c["N"] * c["G"]
    ids = st["page_ids"].long() & 0xFFFFFFFF
    indptr = st["indptr"].long()
    npg = indptr[1:] - indptr[:-1]
    width = -(-st["Tmax"] // P) + 3                     # pages of a unit, at most
    K = torch.zeros((max(ids.numel(), 1), P, D), device=dev)
    V = torch.zeros_like(K)
    rows = torch.zeros(max(ids.numel(), 1), dtype=torch.int64, device=dev)
    for t in range(3):
        mine = (ids >> 30) == t
        page = st["pools"][t][ids[mine] & 0x3FFFFFFF]
        rows[:ids.numel()][mine] = page[:, 0].long() + 256 * page[:, 1].long()
        K[:ids.numel()][mine], V[:ids.numel()][mine] = _rows(t, P, st["lay"], page)
    k = torch.arange(width, device=dev)
    at = (indptr[:-1].unsqueeze(1) + k).clamp(max=max(ids.numel() - 1, 0))
    have = (k < npg.unsqueeze(1)).unsqueeze(-1) & \
        (torch.arange(P, device=dev) < rows[at].unsqueeze(-1))
    have = have.view(U, width * P)
    q = st["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(U, R, D)
    S = torch.bmm(q, K[at].view(U, width * P, D).transpose(1, 2)) / math.sqrt(D)
    if c["cap"]:
        S = c["cap"] * torch.tanh(S / c["cap"])
    slope = qpos = None
    if c["bias"]:
        slope = st["slopes"].view(1, Hkv, 1, G).expand(B, Hkv, N, G).reshape(U, R, 1)
        qpos = st["q_pos"].view(B, 1, N, 1).expand(B, Hkv, N, G).reshape(U, R, 1)
        ro = st["row_of"].view(U, -1).long()
        kpos = torch.zeros((U, width * P + 1), dtype=torch.int32, device=dev)
        where = torch.where(ro >= 0, ro, torch.full_like(ro, width * P))
        kpos.scatter_(1, where, torch.arange(ro.shape[1], device=dev, dtype=torch.int32)
                      .expand(U, -1).contiguous())
        S = S - slope * (qpos - kpos[:, :-1].unsqueeze(1)).float()
    S = S.masked_fill(~have.unsqueeze(1), -math.inf)
    vals = V[at].view(U, width * P, D)
    if c["draft"]:
        kd = st["k"].float().permute(0, 2, 1, 3).reshape(U, N, D)
        vd = st["v"].float().permute(0, 2, 1, 3).reshape(U, N, D)
        Sd = torch.bmm(q, kd.transpose(1, 2)) / math.sqrt(D)
        if c["cap"]:
            Sd = c["cap"] * torch.tanh(Sd / c["cap"])
        if c["bias"]:
            dpos = st["q_pos"].view(B, 1, 1, N).expand(B, Hkv, 1, N).reshape(U, 1, N)
            Sd = Sd - slope * (qpos - dpos).float()
        j = torch.arange(N, device=dev)
        see = ((st["mask"].unsqueeze(-1) >> j) & 1).bool() & (j < st["count"].view(B, 1, 1))
        see = see.view(B, 1, N, 1, N).expand(B, Hkv, N, G, N).reshape(U, R, N)
        S = torch.cat([S, Sd.masked_fill(~see, -math.inf)], -1)
        vals = torch.cat([vals, vd], 1)
    m = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p, vals) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.view(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    live = torch.arange(N, device=dev).view(1, N, 1, 1) < st["count"].view(B, 1, 1, 1)
    st["out"].copy_(torch.where(live, o.to(st["out"].dtype), st["out"]))
    return st["out"]


def _evict(st):
    c, P, B, Hkv, Tmax = st["c"], st["P"], st["B"], st["Hkv"], st["Tmax"]
    U, dev = B * Hkv, st["tier"].device
    tier = st["tier"].view(U, Tmax)
    pos = torch.arange(Tmax, device=dev).view(1, Tmax)
    T = st["seq_lens"].long().view(B, 1).expand(B, Hkv).reshape(U, 1)
    here = (tier < DROP) & (pos < T)
    held = here & ((pos < c["sink"]) | (pos >= T - c["recent"]))
    left = st["keep"].long().view(B, 1).expand(B, Hkv).reshape(U, 1) - held.sum(1, keepdim=True)
    # highest scores first, ties by position
    key = torch.where(here & ~held, st["score"].view(U, Tmax), torch.full((), -1.0, device=dev))
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, pos.expand(U, Tmax).contiguous())
    stay = held | (here & (rank < left))
    new_tier = torch.where(stay, tier, torch.full_like(tier, DROP)).view(B, Hkv, Tmax)
    row_of, tip, pages, n = _tables(new_tier, P, B, Hkv)
    ids, seg = _page_ids(pages, st["free"], st["cursor"].long())
    hdr = _headers(ids, seg, n, P, Hkv, tip)
    old_ids, old_ptr = st["page_ids"].long(), st["indptr"].long()
    unit = torch.arange(U, device=dev).view(U, 1)
    for t in range(3):
        cb = (0, 64, 48)[t]
        pay, stride = _page_bytes(t, P)
        move = (new_tier.view(U, Tmax) == t)
        uu = unit.expand(U, Tmax)[move]
        src, dst = st["row_of"].view(U, Tmax)[move].long(), row_of.view(U, Tmax)[move].long()
        mine = seg % 3 == t
        local = torch.zeros(ids.numel() + 1, dtype=torch.int64, device=dev)
        local[:-1][mine] = torch.arange(int(mine.sum()), device=dev)
        page = torch.zeros((int(mine.sum()), stride), dtype=torch.uint8, device=dev)
        page[:, :16] = hdr[mine].contiguous().view(torch.uint8).view(-1, 16)
        a = (old_ids[old_ptr[uu] + src // P] & 0x3FFFFFFF, src % P)          # slot, row
        b = (local[tip[0::3].long()[uu] + dst // P], dst % P)
        pool = st["pools"][t]
        old, new = pool[:, 16:pay], page[:, 16:pay]
        if t == 0:
            k0, v2 = st["lay"]["k0"].view(P, D), st["lay"]["v2"].view(P, D) + P * D
            oh, nh = pool.view(torch.float16)[:, 8:pay // 2], page.view(torch.float16)[:, 8:pay // 2]
            for at in (k0, v2):
                nh[b[0].unsqueeze(1), at[b[1]]] = oh[a[0].unsqueeze(1), at[a[1]]]
        else:
            j = torch.arange(cb, device=dev)
            spans = (torch.arange(2, device=dev) + 2 * torch.arange(P, device=dev).view(P, 1),
                     2 * P + j + cb * torch.arange(P, device=dev).view(P, 1),
                     (2 + cb) * P + torch.arange(2, device=dev)
                     + 2 * torch.arange(P, device=dev).view(P, 1),
                     (4 + cb) * P + st["lay"]["v1"].view(P, D))
            for at in spans:
                new[b[0].unsqueeze(1), at[b[1]]] = old[a[0].unsqueeze(1), at[a[1]]]
        pool[ids[mine] & 0x3FFFFFFF] = page
    new_ids = st["new"]["ids"]
    new_ids[:ids.numel()] = ids.to(torch.int32)
    return dict(tier=new_tier, row_of=row_of, indptr=tip[0::3].contiguous(), tier_indptr=tip,
                page_ids=new_ids, pools=st["pools"])


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The verification's output in 64 bits, a sequence's head at a time, from
    the bytes of the pages (eviction moves whole values: nothing is rounded)."""
    c = dict(case)
    if c["op"] == "evict":
        return None
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    f64, dev = torch.float64, st["q"].device
    B, Hkv, G, N, P = c["B"], c["Hkv"], c["G"], c["N"], c["P"]
    ids, ptr = st["page_ids"].cpu().tolist(), st["indptr"].cpu().tolist()
    ids = np.array(ids, dtype=np.int64)
    res = torch.zeros((B, N, Hkv * G, D), dtype=f64, device=dev)
    dims = torch.arange(D, device=dev)
    prow = torch.arange(P, device=dev)
    count = st["count"].cpu().tolist()
    mask = None if st["mask"] is None else st["mask"].cpu().numpy().view(np.uint64)

    def keys_values(t, page):
        """By the byte address of every value."""
        n = page.shape[0]
        byte = lambda at: page.gather(1, at.reshape(1, -1).expand(n, -1))  # noqa: E731

        def halves(at):                                   # element -> two bytes
            at = at.reshape(-1)
            two = torch.stack([at, at + 1], 1)
            return byte(two).contiguous().view(torch.float16).to(f64)

        row, d = prow.view(P, 1), dims.view(1, D)
        frag = 4 * (d % 8) + (row % 8) // 2
        inner = 2 * ((d // 8) % 2) + row % 2
        if t == 0:
            K = halves(16 + 256 * row + 16 * ((d // 8) ^ (4 * (row & 1))) + 2 * (d % 8))
            V = halves(16 + 256 * P + 2048 * (row // 8) + 512 * (d // 32) + 16 * frag
                       + 8 * ((d // 16) % 2) + 2 * inner)
            return K.view(n, P, D), V.view(n, P, D)
        cb = 64 if t == 1 else 48
        rad = halves(16 + 2 * prow).view(n, P, 1)
        sc = halves(16 + (2 + cb) * P + 2 * prow).view(n, P, 1)
        pr = dims // 2
        g, j = (pr // 4) % 4, 4 * (pr // 16) + pr % 4
        base = 16 + 2 * P + cb * row
        if t == 1:
            w = byte(base + (16 * g + j).view(1, D)).view(n, P, D).long()
            ang, share, sect = w // 4, w % 4, 64
        else:
            w = byte(base + (8 * g + j // 2).view(1, D)).view(n, P, D).long()
            ang = torch.where(j % 2 == 1, w // 16, w % 16)
            w = byte(base + (32 + 4 * g + j // 4).view(1, D)).view(n, P, D).long()
            share, sect = (w // (4 ** (j % 4))) % 4, 16
        th = ang.to(f64) * (2 * math.pi / sect)
        K = rad * (share + 1).to(f64) / 16 * torch.where(dims % 2 == 0, th.cos(), th.sin())
        v = byte(16 + (4 + cb) * P + 1024 * (row // 8) + 512 * (d // 64) + 16 * frag
                 + 4 * ((d // 16) % 4) + inner).view(n, P, D)
        return K, sc * torch.where(v > 127, v.to(f64) - 256, v.to(f64))

    for b in range(B):
        m = count[b]
        if m == 0:
            continue
        for h in range(Hkv):
            u = b * Hkv + h
            mine = ids[ptr[u]:ptr[u + 1]] & 0xFFFFFFFF
            q = st["q"][b, :m, h * G:(h + 1) * G].to(f64)
            score, val, kpos = [], [], []
            by_row = None
            if c["bias"]:
                by_row = torch.zeros(len(mine) * P + 1, dtype=f64, device=dev)
                ro = st["row_of"][b, h].long()
                p = (ro >= 0).nonzero().view(-1)
                by_row[ro[p]] = p.to(f64)
            for t in range(3):
                of = np.nonzero(mine >> 30 == t)[0]
                if not len(of):
                    continue
                slot = torch.from_numpy(mine[of] & 0x3FFFFFFF).to(dev)
                page = st["pools"][t][slot]
                K, V = keys_values(t, page)
                ok = prow < (page[:, 0].long() + 256 * page[:, 1].long()).view(-1, 1)
                score.append(torch.einsum("ngd,td->ngt", q, K[ok]) / math.sqrt(D))
                val.append(V[ok])
                if by_row is not None:
                    at = torch.from_numpy(of).to(dev).view(-1, 1) * P + prow
                    kpos.append(by_row[at[ok]])
            if c["draft"]:
                score.append(torch.einsum("ngd,td->ngt", q, st["k"][b, :m, h].to(f64))
                             / math.sqrt(D))
                val.append(st["v"][b, :m, h].to(f64))
                if by_row is not None:
                    kpos.append(st["q_pos"][b, :m].to(f64))
            if not score:
                continue
            s = torch.cat(score, -1)
            if c["cap"]:
                s = c["cap"] * torch.tanh(s / c["cap"])
            if c["bias"]:
                far = st["q_pos"][b, :m].to(f64).view(m, 1, 1) - torch.cat(kpos).view(1, 1, -1)
                s = s - st["slopes"][h * G:(h + 1) * G].to(f64).view(1, G, 1) * far
            if c["draft"]:
                see = np.array([[(int(mask[b, i]) >> k) & 1 for k in range(m)] for i in range(m)],
                               dtype=bool)
                s[:, :, s.shape[-1] - m:].masked_fill_(
                    ~torch.from_numpy(see).to(dev).view(m, 1, m), -math.inf)
            v = torch.cat(val, 0)
            if v.shape[0]:
                res[b, :m, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.softmax(s, -1), v)
    return res
