"""The stream argument of the older calls (decode, append, retier): outputs,
workspaces, cursors and release lists that a call makes itself are made on its
stream, whatever is queued on the current one."""
import numpy as np
import pytest
import torch

from long_context_decode_ada_b200 import skv
from long_context_decode_ada_b200 import workloads as wl
from test_gpu_call_streams import busy
from test_gpu_retier import Window

pytestmark = pytest.mark.gpu


def test_decode_workspaces():
    lens = [9000, 700]
    w = wl.custom(131, 2, 2, 4, 64, lens, wl.MODE_QUOTA, quota=[[T // 10, T // 2, T // 4] for T in lens])
    ctx = skv.Context(64, deterministic=True)
    dev = skv.workload_to_device(w)
    cache = skv.build_cache(ctx, w, dev)
    cache.check()
    want, want_lse = cache.decode(dev["q"], dev["q_dtype"], w.Hq)
    util = torch.zeros((2, 2, 9000), device="cuda")
    cache.decode_utility(dev["q"], dev["q_dtype"], w.Hq, dev["seq_lens"], util)
    n = cache.workspace(w.Hq).numel()
    m = cache.utility_workspace(w.Hq).numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs, utils = [], [torch.zeros_like(util) for _ in range(10)]
    torch.cuda.synchronize()
    for i in range(10):
        outs.append(cache.decode(dev["q"], dev["q_dtype"], w.Hq, stream=side))
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        cache.decode_utility(dev["q"], dev["q_dtype"], w.Hq, dev["seq_lens"], utils[i], stream=side)
        torch.empty(m, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    cache.check()
    for out, lse in outs:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    for u in utils:
        assert torch.equal(u, util)


def test_append_and_retier():
    # the same cycle twice: on the current stream, and on another with the current
    # one busy.  Nothing of the second is made before it
    def cycle(stream):
        x = Window(5, 2, 2, 16, 400, 24, 64, 0.3)
        c, dev = x.cache, x.dev
        demote = torch.zeros((2, 2, x.w.Tmax), dtype=torch.uint8, device="cuda")
        demote[:, :, x.T - 64:x.T - 40] = 1
        budget = torch.tensor([int(0.3 * (x.T + 24) * 2 * 512)] * 2, dtype=torch.int64, device="cuda")
        K = [dev["K"][:, :, x.T + i].contiguous() for i in range(24)]
        V = [dev["V"][:, :, x.T + i].contiguous() for i in range(24)]
        torch.cuda.synchronize()
        keep = busy() if stream is not None else None
        for i in range(24):
            c.append(K[i], V[i], x.seq, stream=stream)
        released, n = c.retier(dev["utility"], demote, budget, x.seq, stream=stream)
        torch.cuda.synchronize()
        c.check()
        del keep
        n = int(n)
        ptr = c.page_indptr.cpu().numpy()
        return (c.tier.cpu().numpy(), c.row_of.cpu().numpy(), ptr, c.page_ids[:ptr[-1]].cpu().numpy(),
                c.free_cursor().cpu().numpy(), np.sort(released[:n].cpu().numpy()))

    a, b = cycle(None), cycle(torch.cuda.Stream())
    assert len(a[-1]) > 0
    for x, y in zip(a, b):
        assert np.array_equal(x, y)
