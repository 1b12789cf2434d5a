"""GPU: attaching and detaching the page bounds waits for what still uses a buffer."""
import pytest
import torch

import workloads as W
from _gpu_common import gpu_ready, to_c_policies
from test_gpu_decode_select import _check_bounds, _keys, _mk

pytestmark = pytest.mark.gpu

POLS = [W.HeadPolicy(W.GLOBAL)] * 2


def _work_ahead(c, stream, busy):
    """A write, a decode and the release of a sequence, queued on `stream` behind a long pass."""
    k = _keys(200, 2, 64, 1)
    q = W.normal((1, 4, 64), 9, device="cuda")
    for passes in (0, 40):                                      # (once without: kernels are loaded at their first launch)
        c.set_policy(0, to_c_policies([POLS]))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(passes):
                busy.add_(1.0)
            c.build(0, 0, k, k)
            c.decode_select(0, [0], q, 2)
            c.release(0)
    assert not stream.query()                                   # (40 passes over 2 GiB take longer than this)
    return k, q


@pytest.mark.parametrize("again", [False, True])
def test_a_buffer_is_not_let_go_while_it_is_used(again):
    """Detached, or replaced by another: nothing is on its way when the call returns."""
    import head_aware_paged_gb300 as H
    gpu_ready()
    c = _mk(4, 2, 64, 16, 1, 300)
    busy, s = torch.zeros(1 << 28, device="cuda"), torch.cuda.Stream()
    k, q = _work_ahead(c, s, busy)
    if again:
        c.attach_page_bounds()
    else:
        H.sp_attach_page_bounds(c.handle, None)
    assert s.query()
    if not again:
        c.attach_page_bounds()
    c.set_policy(0, to_c_policies([POLS]))
    c.build(0, 0, k, k)
    _check_bounds(c, [0], [0, 1])
    c.decode_select(0, [0], q, 2)
    assert c.status() == 0


def test_the_same_buffer_again():
    """Cleared for its next use after the earlier calls, not under them."""
    import head_aware_paged_gb300 as H
    gpu_ready()
    c = _mk(4, 2, 64, 16, 1, 300)
    busy, s = torch.zeros(1 << 28, device="cuda"), torch.cuda.Stream()
    _work_ahead(c, s, busy)
    H.sp_attach_page_bounds(c.handle, c._bounds)
    torch.cuda.synchronize()
    codes, step = c.page_bounds()
    assert not codes.any() and not step.any()


def test_without_bounds():
    """Before they are attached and after they are detached: refused, and writes go on."""
    import head_aware_paged_gb300 as H
    gpu_ready()
    c = _mk(4, 2, 64, 16, 1, 300, attach=False)
    c.set_policy(0, to_c_policies([POLS]))
    k, q = _keys(200, 2, 64, 1), W.normal((1, 4, 64), 9, device="cuda")
    for _ in range(2):
        with pytest.raises(RuntimeError):
            c.page_bounds()
        c.build(0, 0, k, k)
        with pytest.raises(H.SegPagedError):
            c.decode_select(0, [0], q, 2)
        c.release(0)
        c.attach_page_bounds()
        c.build(0, 0, k, k)
        _check_bounds(c, [0], [0, 1])
        with pytest.raises(H.SegPagedError):                    # tokens held
            c.detach_page_bounds()
        c.page_bounds()
        c.release(0)
        c.detach_page_bounds()
    assert c.status() == 0
