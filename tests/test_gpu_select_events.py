"""GPU: the launch events of the decode over chosen pages lie around its kernels: after
what the stream held before the call, before what it got afterwards, once a call."""
import pytest
import torch

import workloads as W
from _gpu_common import gpu_ready, to_c_policies
from test_gpu_decode_select import _keys, _mk

pytestmark = pytest.mark.gpu


def _one_long(top):
    """One unit of 2,438 pages: the choice in the decode's launch (few pages kept), or
    in one of its own (more than a block's memory holds)."""
    c = _mk(4, 1, 64, 16, 1, 40000)
    c.set_policy(0, to_c_policies([[W.HeadPolicy(W.GLOBAL)]]))
    k = _keys(39000, 1, 64, 1)
    c.build(0, 0, k, k)
    return c, [0], W.normal((1, 4, 64), 9, device="cuda"), top


def _one_heavy_among_many():
    """512 units, one of them with 270 kept pages: they would fit a block's memory, and
    the launcher hands the call to the two launches all the same."""
    c = _mk(8, 8, 64, 16, 64, 6000, pages=6000)
    k = _keys(5000, 8, 64, 1)
    for s in range(64):
        first = W.HeadPolicy(W.GLOBAL) if s == 0 else W.HeadPolicy(W.LOCAL, 2, 9)
        c.set_policy(s, to_c_policies([[first] + [W.HeadPolicy(W.LOCAL, 2, 9)] * 7]))
        n = 5000 if s == 0 else 40
        c.build(s, 0, k[:n], k[:n])
    return c, list(range(64)), W.normal((64, 8, 64), 9, device="cuda"), 266


CASES = {"one launch": lambda: _one_long(3), "two launches": lambda: _one_long(2100), "handed on": _one_heavy_among_many}


@pytest.mark.parametrize("case", list(CASES))
def test_launch_events_lie_around_the_kernels(case):
    gpu_ready()
    c, ids, q, top = CASES[case]()
    busy = torch.zeros(1 << 28, device="cuda")                  # 1 GiB: a pass over it takes longer than the decode
    want = c.decode_select(0, ids, q, top, 1, 3)
    inner, outer = ([torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in range(2))
    for x in inner:
        x.record()                                              # (makes the events; stale unless the call records them)
    torch.cuda.synchronize()
    c.set_launch_events(*inner)
    busy.add_(1.0)
    outer[0].record()
    got = c.decode_select(0, ids, q, top, 1, 3, out=torch.empty_like(want[0]), lse=torch.empty_like(want[1]),
                          pages=torch.empty_like(want[2]))
    outer[1].record()
    busy.add_(1.0)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # (the clock's steps are below a microsecond; the host has queued the call while `busy` runs)
    before, span, after = (a.elapsed_time(b) for a, b in ((outer[0], inner[0]), inner, (inner[1], outer[1])))
    whole = outer[0].elapsed_time(outer[1])
    assert before >= -1e-3 and after >= -1e-3, (before, after)
    assert 0.5 * whole <= span <= whole + 1e-3 and span > 2e-3, (span, whole)
    # one call: the next leaves the pair where it was
    c.decode_select(0, ids, q, top, 1, 3)
    torch.cuda.synchronize()
    assert inner[0].elapsed_time(inner[1]) == span


def test_a_refused_call_records_nothing():
    """Armed events keep what they held when the call is refused, and stay armed."""
    import head_aware_paged_gb300 as H
    gpu_ready()
    c = _mk(4, 1, 64, 16, 2, 40000)
    for s in range(2):
        c.set_policy(s, to_c_policies([[W.HeadPolicy(W.GLOBAL)]]))
    k = _keys(39000, 1, 64, 1)
    c.build(0, 0, k, k)
    q = W.normal((2, 4, 64), 9, device="cuda")
    inner = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    inner[0].record()
    torch.zeros(1 << 26, device="cuda").add_(1.0)
    inner[1].record()
    torch.cuda.synchronize()
    was = inner[0].elapsed_time(inner[1])
    c.set_launch_events(*inner)
    for top in (3, 2100):
        with pytest.raises(H.SegPagedError):
            c.decode_select(0, [0, 1], q, top)                  # sequence 1 is empty
    torch.cuda.synchronize()
    assert inner[0].elapsed_time(inner[1]) == was
    c.decode_select(0, [0], q[:1].contiguous(), 3)
    torch.cuda.synchronize()
    assert inner[0].elapsed_time(inner[1]) != was
