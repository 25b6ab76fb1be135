"""A paged store read back from its bytes in 64 bits: for every unit the
resident rows' keys, values, tiers and positions, by the documented page
layout (one value at a time, without the library's tables)."""
import numpy as np

D = 128
LLOYD = np.array([383, 807, 1249, 1831]) / 1024 / 8


def _v_offset(row, d, size):
    frag = 4 * (d % 8) + (row % 8) // 2
    e = 2 * ((d // 8) % 2) + row % 2
    if size == 1:
        return 1024 * (row // 8) + 512 * (d // 64) + 16 * frag + 4 * ((d // 16) % 4) + e
    return 2048 * (row // 8) + 512 * (d // 32) + 16 * frag + 8 * ((d // 16) % 2) + 2 * e


def page_rows(page, tier, P, t1_53=False, lloyd=False):
    """fp64 (keys, values) [P][128] of one page's bytes."""
    row = np.arange(P)[:, None]
    d = np.arange(D)[None, :]
    half = lambda at: (page[at].astype(np.uint16) | (page[at + 1].astype(np.uint16) << 8)).view(  # noqa: E731
        np.float16).astype(np.float64)
    if tier == 0:
        K = half(16 + 256 * row + 16 * ((d // 8) ^ (4 * (row & 1))) + 2 * (d % 8))
        return K, half(16 + 256 * P + _v_offset(row, d, 2))
    cb = 64 if tier == 1 else 48
    r = half(16 + 2 * np.arange(P))[:, None]
    sc = half(16 + (2 + cb) * P + 2 * np.arange(P))[:, None]
    pr = d // 2
    g, j = (pr // 4) % 4, 4 * (pr // 16) + pr % 4
    base = 16 + 2 * P + cb * row
    levels = LLOYD if lloyd else (np.arange(4) + 1) / 16
    if tier == 1:
        w = page[base + 16 * g + j].astype(np.int64)
        if t1_53:
            ang, share, bits = w >> 3, ((w & 7) + 1) / 32, 5
        else:
            ang, share, bits = w >> 2, levels[w & 3], 6
    else:
        ang = (page[base + 8 * g + j // 2].astype(np.int64) >> (4 * (j % 2))) & 15
        share = levels[(page[base + 32 + 4 * g + j // 4].astype(np.int64) >> (2 * (j % 4))) & 3]
        bits = 4
    th = ang * (2 * np.pi / (1 << bits))
    K = r * share * np.where(d % 2 == 0, np.cos(th), np.sin(th))
    V = sc * page[16 + (4 + cb) * P + _v_offset(row, d, 1)].view(np.int8).astype(np.float64)
    return K, V


def read_store(cache, t1_53=False, lloyd=False):
    """Per unit a dict: K, V fp64 [n][128], tier [n], row [n] (local row),
    pos [n] (the token at that row by the row map, -1: none)."""
    P = cache.ctx.P
    ptr = cache.page_indptr.cpu().numpy()
    ids = cache.page_ids.cpu().numpy().view(np.uint32)
    pools = [p.cpu().numpy() for p in cache.pools]
    row_of = cache.row_of.cpu().numpy().reshape(cache.B * cache.Hkv, -1)
    units = []
    for u in range(cache.B * cache.Hkv):
        K, V, tier, row = [np.zeros((0, D))], [np.zeros((0, D))], [], []
        for k, g in enumerate(range(ptr[u], ptr[u + 1])):
            t, slot = int(ids[g]) >> 30, int(ids[g]) & 0x3FFFFFFF
            page = pools[t][slot * cache.stride[t]: slot * cache.stride[t] + cache.payload[t]]
            n = int(page[0]) + 256 * int(page[1])
            assert page[2] == t and page[3] == 0x5A and n <= P
            a, b = page_rows(page, t, P, t1_53, lloyd)
            K.append(a[:n])
            V.append(b[:n])
            tier += [t] * n
            row += [k * P + r for r in range(n)]
        row = np.array(row, dtype=np.int64)
        at = np.full(int(ptr[u + 1] - ptr[u]) * P + 1, -1, dtype=np.int64)
        ok = row_of[u] >= 0
        at[row_of[u][ok]] = np.nonzero(ok)[0]
        units.append(dict(K=np.concatenate(K), V=np.concatenate(V), tier=np.array(tier, np.int64),
                          row=row, pos=at[row] if len(row) else row))
    return units


def tree_reference(cache, q, k=None, v=None, mask=None, count=None, softcap=0.0, slopes=None,
                   q_pos=None, t1_53=False, lloyd=False):
    """fp64 (out, lse, out bound, lse bound) of the tree attention.

    The bounds count the roundings of the kernels.  A coded key component is
    a table entry rounded to fp16 times the radius rounded to fp16 (2 * 2^-11
    relative), T0 and drafted keys are exact; products add up in fp32 (2^-18
    of their absolute sum covers 128 terms in any order); capped and biased
    scores are fp32 (2^-20 relative to their parts, 1e-5 for the tanh): eps_t
    bounds the change of score t.  A change of scores moves the output by at
    most sum p eps |v| + (sum p eps)(sum p |v|) to first order (5% for the
    rest); weights and coded values are rounded to fp16 once more each
    (2 * 2^-11, and 2^-25 absolute against a largest weight of at least 1);
    the output to its own type."""
    B, N, Hq, _ = q.shape
    Hkv = cache.Hkv
    G = Hq // Hkv
    units = read_store(cache, t1_53, lloyd)
    out = np.zeros((B, N, Hq, D))
    lse = np.full((B, N, Hq), -np.inf)
    ob, lb = np.zeros_like(out), np.zeros_like(lse)
    half = 2.0 ** -8 if str(q.dtype) == "torch.bfloat16" else 2.0 ** -11
    f = lambda x: x.detach().cpu().double().numpy()  # noqa: E731
    qn = f(q)
    kn = None if k is None else f(k)
    vn = None if v is None else f(v)
    for b in range(B):
        n = N if count is None else int(count[b])
        for i in range(n):
            for hq in range(Hq):
                h = hq // G
                s = units[b * Hkv + h]
                K, V = s["K"], s["V"]
                coded = s["tier"] > 0
                pos = s["pos"]
                if kn is not None:
                    js = [j for j in range(n) if (j <= i if mask is None else
                                                  (int(mask[b, i]) >> j) & 1)]
                    K = np.concatenate([K, kn[b, js, h]])
                    V = np.concatenate([V, vn[b, js, h]])
                    coded = np.concatenate([coded, np.zeros(len(js), bool)])
                    if q_pos is not None:
                        pos = np.concatenate([pos, [int(q_pos[b, j]) for j in js]])
                if not len(K):
                    continue
                x = (K @ qn[b, i, hq]) / np.sqrt(D)
                ab = (np.abs(K) @ np.abs(qn[b, i, hq])) / np.sqrt(D)
                eps = ab * np.where(coded, 2.0 ** -10, 0.0) + ab * 2.0 ** -18 + 1e-6
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                    eps = eps + 1e-5 + np.abs(x) * 2.0 ** -20
                if slopes is not None:
                    far = float(slopes[hq]) * (int(q_pos[b, i]) - pos)
                    x = x - far
                    eps = eps + (np.abs(far) + np.abs(x)) * 2.0 ** -20
                m = x.max()
                p = np.exp(x - m)
                l = p.sum()
                p /= l
                out[b, i, hq] = p @ V
                lse[b, i, hq] = m + np.log(l)
                A = p @ np.abs(V)
                pe = p @ eps
                ob[b, i, hq] = (1.05 * ((p * eps) @ np.abs(V) + pe * A) + 2.2 * 2.0 ** -11 * A
                                + len(x) * 2.0 ** -25 * np.abs(V).max(0)
                                + half * np.abs(out[b, i, hq]) + 1e-7)
                ob[b, i, hq] *= 1 + half
                lb[b, i, hq] = 1.05 * pe + 2.0 ** -20 * abs(lse[b, i, hq]) + 1e-5
    return out, lse, ob, lb
