"""Tree attention: caps without bias and values beyond fp16 in every form, calls
that follow each other on one workspace, and captured calls whose drafted
values change size."""
import pytest
import torch

from long_context_decode_ada_b200 import skv
from test_gpu_tree import compare, drafts, make_store

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [9, 16, 17, 24, 32])      # 36 to 128 rows a kv head
@pytest.mark.parametrize("cap", [2.0, 20.0, 128.0, 500.0, 1e6])
def test_caps_without_bias(N, cap):
    cache, _ = make_store([700, 90, 0], 1, 4, 32, seed=101, k_scale=4.0)
    q, k, v, par = drafts(3, N, 1, 4, 61)
    q[:, :, 0] *= 8
    mask = skv.tree_mask(par)
    lse = torch.empty((3, N, 4), device="cuda")
    for splits in (1, 0):
        got = cache.tree_attention(q, k, v, mask=mask.cuda(), softcap=cap, lse=lse, num_splits=splits)
        compare(cache, got, q, k=k, v=v, mask=mask, softcap=cap)


@pytest.mark.parametrize("N", [1, 2, 3, 5, 8, 12, 33, 64])
@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0), dict(bias=True), dict(softcap=400.0, bias=True)])
def test_values_beyond_fp16_in_every_form(N, kw):
    lens = [130, 0]
    cache, dev = make_store(lens, 1, 4, 16, seed=103)
    q, k, v, _ = drafts(2, N, 1, 4, 63, torch.bfloat16, torch.bfloat16)
    v[0, 0, 0, 9], v[1, N // 2, 0, 64], v[1, N - 1, 0, 127] = 9e4, -1e7, 3e5
    kw = dict(kw)
    extra = {}
    if kw.pop("bias", False):
        kw["slopes"] = torch.tensor([0.1, 0.02, 0.5, 0.0], device="cuda")
        kw["q_pos"] = (dev["seq_lens"][:, None] + torch.arange(N, device="cuda")[None]).to(torch.int32)
        extra["seq_lens"] = dev["seq_lens"]
    lse = torch.empty((2, N, 4), device="cuda")
    got = cache.tree_attention(q, k, v, lse=lse, **kw, **extra)
    compare(cache, got, q, k=k, v=v, **kw)


@pytest.mark.parametrize("N", [2, 12, 40])
def test_calls_one_after_another_on_one_workspace(N):
    # each with values of another size: what one call leaves in the workspace is
    # not the next one's
    cache, _ = make_store([500, 60], 1, 4, 16, seed=107)
    q, k, v, _ = drafts(2, N, 1, 4, 65, torch.bfloat16, torch.bfloat16)
    ws = cache.tree_workspace(N, 4)
    sizes = [2.0 ** -e for e in (0, 9, 20, 3, 14, 0, 30)]
    vs = [v * s for s in sizes]
    want = []
    for x in vs:
        want.append(cache.tree_attention(q, k, x)[0])
        torch.cuda.synchronize()
    outs = [cache.tree_attention(q, k, x, workspace=ws)[0] for _ in range(3) for x in vs]
    cache.check()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % len(vs)])


@pytest.mark.parametrize("N,bias", [(4, True), (20, False), (20, True), (40, False)])
def test_captured_calls_follow_the_values_sizes(N, bias):
    cache, dev = make_store([400, 33], 1, 4, 16, seed=109)
    q, k, v, _ = drafts(2, N, 1, 4, 67, torch.bfloat16, torch.bfloat16)
    kw = {}
    if bias:
        kw = dict(slopes=torch.tensor([0.1, 0.02, 0.5, 0.0], device="cuda"), seq_lens=dev["seq_lens"],
                  q_pos=(dev["seq_lens"][:, None] + torch.arange(N, device="cuda")[None]).to(torch.int32))
    v0 = v.clone()
    out = torch.zeros_like(q)
    ws = cache.tree_workspace(N, 4, positions=bias)
    cache.tree_attention(q, k, v, out=out, workspace=ws, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.tree_attention(q, k, v, out=out, workspace=ws, **kw)
    for e in (0, 12, 25, 0):
        v.copy_(v0 * 2.0 ** -e)
        graph.replay()
        torch.cuda.synchronize()
        want, _ = cache.tree_attention(q, k, v, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        ref = {n: x for n, x in kw.items() if n != "seq_lens"}
        compare(cache, (out, None), q, k=k, v=v, **ref)
