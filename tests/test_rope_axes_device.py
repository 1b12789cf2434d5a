"""CPU: sp_rope_axes takes tensors of the current CUDA device and no others (the
library launches there, whatever the addresses are; a launch on host memory or on
another GPU's would return before that memory's own work, or fault).  No refused call
gets as far as the library."""
import pytest
import torch

import head_aware_paged_gb300 as H


class On(torch.Tensor):
    """A CPU tensor that says it lies on CUDA device `index`."""
    index = 0

    def get_device(self):
        return self.index


def _on(x, index):
    y = x.as_subclass(On)
    y.index = index
    return y


class Reached(Exception):
    pass


@pytest.fixture
def library(monkeypatch):
    """The library is not called: a call that gets there raises Reached.  Device 0 is current."""
    def load():
        raise Reached
    monkeypatch.setattr(H, "load", load)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def _args(index=None, rows=3, heads=2, d=64):
    x, p = torch.zeros(rows, heads, d, dtype=torch.bfloat16), torch.zeros(3, rows, dtype=torch.int64)
    return (x, p) if index is None else (_on(x, index), _on(p, index))


@pytest.mark.parametrize("side", ["q", "k", "both"])
def test_host_memory_is_refused(library, side):
    x, p = _args()
    with pytest.raises(AssertionError):
        H.sp_rope_axes(x if side != "k" else None, x.clone() if side != "q" else None, p, [0] * 32)


def test_another_device_is_refused(library):
    x, p = _args(1)
    out = _on(torch.zeros(3, 2, 64, dtype=torch.bfloat16), 1)
    for kw in (dict(), dict(stream=0)):
        with pytest.raises(AssertionError):
            H.sp_rope_axes(x, None, p, [0] * 32, q_out=out, **kw)
        with pytest.raises(AssertionError):
            H.sp_rope_axes(None, x, p, [0] * 32, k_out=out, **kw)


def test_devices_that_differ_are_refused(library):
    """Queries on the current device; keys, positions or an output elsewhere."""
    x, p = _args(0)
    out = _on(torch.zeros(3, 2, 64, dtype=torch.bfloat16), 0)
    away, p_away = _args(1)
    host, p_host = _args()
    for bad in (dict(k=away), dict(k=host), dict(axis_pos=p_away), dict(axis_pos=p_host), dict(q_out=away), dict(q_out=host)):
        a = dict(q=x, k=None, axis_pos=p, axis_of=[0] * 32, q_out=out, k_out=out)
        a.update(bad)
        with pytest.raises(AssertionError):
            H.sp_rope_axes(**a)


def test_the_current_device_is_taken(library):
    x, p = _args(0)
    with pytest.raises(Reached):
        H.sp_rope_axes(x, None, p, [0] * 32, q_out=_on(torch.zeros(3, 2, 64, dtype=torch.bfloat16), 0), stream=0)
