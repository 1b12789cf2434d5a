"""GPU: the decode over chosen pages in two launches (the choice in one of its own)
under capture and replay, where graphs and eager calls share its tickets, scores and
table of kept pages."""
import pytest
import torch

import workloads as W
from _gpu_common import gpu_ready, to_c_policies
from test_gpu_decode_select import _check_select, _keys, _mk

pytestmark = pytest.mark.gpu

G, L = W.GLOBAL, W.LOCAL


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_two_graphs_and_an_eager_call_in_two_launches(kv):
    """More than 2,048 kept pages, or more than 4,096 candidates: neither fits a block's
    memory.  Replays in both orders with an eager call between, all of them the bits
    of the first calls; then other queries in the graphs, against the oracle."""
    gpu_ready()
    hq, hkv, d, P = 8, 2, 128, 16
    lens = [70000, 36000, 500]
    pols = [W.HeadPolicy(G), W.HeadPolicy(L, 4, 60)]
    c = _mk(hq, hkv, d, P, 3, 70016, kv=kv, pages=sum(n // P + 2 for n in lens) + 3 * 8)
    for s, n in enumerate(lens):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(n, hkv, d, s), W.normal((n, hkv, d), s + 5, device="cuda"))
    # (sequences, top, first, newest): candidates past 4,096; kept pages past 2,048
    calls = [([0, 2], 20, 1, 2), ([1, 0], 2060, 0, 3), ([1], 2100, 2, 2)]
    qs = [W.normal((len(ids), hq, d), 9 + i, device="cuda") for i, (ids, _, _, _) in enumerate(calls)]
    want = [c.decode_select(0, ids, q, *a) for q, (ids, *a) in zip(qs, calls)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q, (ids, *a) in list(zip(qs, calls))[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.decode_select(0, ids, q, *a))
        graphs.append(g)
    for turn in range(4):
        for x in outs:
            for t in x:
                t.zero_()
        got = None
        for g in graphs if turn % 2 == 0 else graphs[::-1]:
            g.replay()
            if got is None:
                got = c.decode_select(0, calls[2][0], qs[2], *calls[2][1:])
        torch.cuda.synchronize()
        for a, b in zip(outs + [got], want):
            for x, y in zip(a, b):
                assert torch.equal(x, y), turn
    for q in qs[:2]:
        q.copy_(W.normal(tuple(q.shape), 40, device="cuda"))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for q, (ids, *a), res in zip(qs, calls, outs):
        _check_select(c, ids, pols, q, *a, what="replay", res=tuple(t.clone() for t in res))
