"""GPU: rotation at positions far beyond 2^31, by frequencies of both signs, against
exact angles.

The angle is off by |p| (2^-65 + |w| 2^-55) turns (the frequency's fraction of a turn)
and 2^-33 (its own rounding); the rest as in test_gpu_rope_axes: half a bf16 step of the
value and 2^-21 of the rotated pair."""
import numpy as np
import pytest
import torch

import workloads as W
from _angles import turns
from _gpu_common import f64, gpu_ready, to_c_policies
from test_gpu_rope_axes import _mk

pytestmark = pytest.mark.gpu

POSITIONS = [s * ((1 << e) + o) for e in (20, 33, 40, 44, 48, 50, 52) for s, o in ((1, 3), (-1, 12345))]


def _turned(x, pos, freq):
    x = f64(x)
    half = x.shape[-1] // 2
    t = np.array([[float(turns(w, p)) for w in freq] for p in pos])[:, None]
    c, s = np.cos(2 * np.pi * t), np.sin(2 * np.pi * t)
    y = np.concatenate([x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s], -1)
    p, w = np.abs(np.array(pos, np.float64))[:, None, None], np.abs(np.array(freq))[None, None]
    angle = 2 * np.pi * (p * (2.0 ** -65 + w * 2.0 ** -55) + 2.0 ** -33)
    pair = np.hypot(x[..., :half], x[..., half:]) * (2.0 ** -21 + angle)
    return y, 2.0 ** -8 * np.abs(y) + np.concatenate([pair, pair], -1) + 1e-30


@pytest.mark.parametrize("sign", [1, -1, 0])                   # 0: both in turn
@pytest.mark.parametrize("d", [64, 128])
def test_far_positions(d, sign):
    import head_aware_paged_gb300 as H
    gpu_ready()
    rng = np.random.default_rng(d)
    w = 2.0 ** rng.uniform(-32, -6, d // 2)
    freq = [float(x) * (sign or (1 if i % 2 else -1)) for i, x in enumerate(w)]
    n = len(POSITIONS)
    q, k = W.normal((n, 3, d), 5, device="cuda"), W.normal((n, 2, d), 6, device="cuda")
    p = torch.tensor([POSITIONS], device="cuda")
    got = H.sp_rope_axes(q, k, p, [0] * (d // 2), inv_freq=freq)
    for a, x in zip(got, (q, k)):
        ref, tol = _turned(x, POSITIONS, freq)
        worst = (np.abs(f64(a) - ref) / tol).max()
        assert worst <= 1.0, worst
    # the opposite positions by the opposite frequencies: the same angles, bit for bit
    back = H.sp_rope_axes(q, k, -p, [0] * (d // 2), inv_freq=[-x for x in freq])
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    # and on the way into the pages
    c = _mk(2, 2, d, 16, 1, 64, 16)
    c.set_policy(0, to_c_policies([[W.HeadPolicy(W.GLOBAL)] * 2]))
    qr = c.append_kv_rope_axes(0, [0], [0, n], q[:, :2], k, k, p, [0] * (d // 2), inv_freq=freq)
    assert torch.equal(qr, got[0][:, :2])
    for h in range(2):
        ids, at = c.export_table(0, 0, h)
        rows = c.k_pool()[torch.tensor(ids, device="cuda")].reshape(-1, d)[:n]
        assert torch.equal(rows, got[1][:, h])
