"""The workspaces of the tree attention and the eviction lie where the store's
pools lie, whatever device is the current one (a store made for "cuda", with
no index, keeps the device it was made on)."""
import torch

from long_context_decode_ada_b200 import skv


def test_workspaces_follow_the_pools():
    cache = skv.PagedCache(skv.Context(16), 2, 2, 64, [4, 4, 4], device="cpu")
    # what an allocation on "cuda" without an index gives after another device
    # has become the current one
    cache.device = torch.device("meta")
    assert cache.tree_workspace(4, 8).device == cache.pools[0].device
    assert cache._evict_workspace().device == cache.pools[0].device
