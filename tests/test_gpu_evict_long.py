"""Eviction of long sequences with protected tokens and unusual scores: the
select with its positions in registers (up to 131072) and the one beyond."""
import pytest
import torch

from test_gpu_evict import check_eviction, make_store, scores

pytestmark = pytest.mark.gpu


def expected(tier, s, keep, lens, sink, recent, prot):
    """The tiers that stay, by a stable sort; NaN below everything."""
    want = torch.full_like(tier, 3)
    T = tier.shape[2]
    pos = torch.arange(T)
    for b, L in enumerate(lens):
        res = (tier[b, 0] < 3) & (pos < L)
        held = res & ((pos < sink) | (pos >= L - recent) | (prot[b, 0] > 0))
        cand = torch.nonzero(res & ~held).view(-1)
        x = s[b, 0][cand].double()
        low = torch.isnan(x)
        # NaN last: by the number, then behind it
        order = torch.argsort(torch.where(low, torch.full_like(x, -float("inf")), x), descending=True,
                              stable=True)
        order = torch.cat([order[~low[order]], order[low[order]]])
        stay = held.clone()
        stay[cand[order[:max(0, int(keep[b]) - int(held.sum()))]]] = True
        want[b, 0] = torch.where(stay, tier[b, 0], want[b, 0])
    return want


@pytest.mark.parametrize("T", [9000, 40000, 131072, 140001])
@pytest.mark.parametrize("kind", ["plain", "odd"])
def test_protected_tokens_of_long_sequences(T, kind):
    lens = [T, T // 2 + 1]
    cache, dev = make_store(lens, 1, 1, 64, f=(0.02, 0.3, 0.5), seed=T % 89)
    s = scores((2, 1, T), 7, zeros=0.3)
    s = (s * 16).round() / 16
    if kind == "odd":
        s[..., 1::7] = float("nan")
        s[..., 2::11] = -float("inf")
        s[..., 3::13] = float("inf")
        s[..., 5::17] = -0.0
        s[..., 4::5] *= -1
    g = torch.Generator().manual_seed(T)
    prot = (torch.rand((2, 1, T), generator=g) < 0.1).to(torch.uint8)
    tier = cache.tier.cpu()
    for keep in ([T // 2, 100], [T // 20, T // 3], [T, 0]):
        kd = torch.tensor(keep, dtype=torch.int32)
        new = cache.evict(s.cuda(), dev["seq_lens"], kd.cuda(), sink=5, recent=40, protect=prot.cuda())
        check_eviction(cache, new, expected(tier, s, keep, lens, 5, 40, prot).numpy(), dev)
