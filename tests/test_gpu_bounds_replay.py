"""GPU: page bounds after replays of captured writes, whatever the heads were when
the write was captured.  Bounds equal the oracle's bit for bit."""
import numpy as np
import pytest
import torch

import workloads as W
from _gpu_common import gpu_ready, to_c_policies
from test_gpu_decode_select import _check_bounds, _check_select, _keys, _mk

pytestmark = pytest.mark.gpu

G, L, R = W.GLOBAL, W.LOCAL, W.RETRIEVAL


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("axes", [False, True])
def test_heads_became_global_after_the_capture(kv, axes):
    """Captured while no head is GLOBAL; the sequence is released, its heads become
    GLOBAL, it is filled past the captured token, and the replay writes into a full
    page: its bounds follow the new key."""
    gpu_ready()
    hq, hkv, d, P = 4, 2, 128, 16
    c = _mk(hq, hkv, d, P, 2, 300, kv=kv)
    before = [W.HeadPolicy(L, 2, 64), W.HeadPolicy(R, idx=np.arange(0, 60, 3, dtype=np.int32))]
    after = [W.HeadPolicy(G), W.HeadPolicy(G)]
    for s in range(2):
        c.set_policy(s, to_c_policies([before]))
        c.build(s, 0, _keys(41 + s, hkv, d, s), W.normal((41 + s, hkv, d), s + 5, device="cuda"))
    x = W.normal((2, hq + 2 * hkv, d), 9, device="cuda")
    q, k, v = x[:, :hq].contiguous(), x[:, hq:hq + hkv].contiguous(), x[:, hq + hkv:].contiguous()
    p = torch.zeros(3, 2, dtype=torch.int64, device="cuda")
    qr = torch.empty_like(q)

    def write():
        if axes:
            c.append_kv_rope_axes(0, [0, 1], [0, 1, 2], q, k, v, p, [0] * 64, pos=[39, 40], q_out=qr)
        else:
            c.append_kv_rope(0, [0, 1], [0, 1, 2], q, k, v, pos=[39, 40], q_out=qr)

    write()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        write()
    for s in range(2):
        c.release(s)
        c.set_policy(s, to_c_policies([after]))
        c.build(s, 0, _keys(100 + s, hkv, d, 10 + s), W.normal((100 + s, hkv, d), 15, device="cuda"))
    _check_bounds(c, [0, 1], [0, 1])
    k.copy_(W.normal((2, hkv, d), 20, device="cuda") * 9)          # larger than any key there
    g.replay()
    torch.cuda.synchronize()
    _check_bounds(c, [0, 1], [0, 1])
    _check_select(c, [0, 1], after, q, 2, 1, 1, what="after the replay")
    # and as LOCAL and RETRIEVAL heads again, the replay computes none
    for s in range(2):
        c.release(s)
        c.set_policy(s, to_c_policies([before]))
        c.build(s, 0, _keys(50, hkv, d, 30), W.normal((50, hkv, d), 31, device="cuda"))
    bounds = [t.clone() for t in c.page_bounds()]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bounds, c.page_bounds())) and c.status() == 0
