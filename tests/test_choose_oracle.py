"""Pins of the page-choice oracle (CPU), and the refusals of the calls around it
that need no device."""
import ctypes

import numpy as np
import pytest

from oracle import choose


def test_grid_is_the_least_power_of_two():
    for a, e in ((127.0, 0), (127.0001, 1), (128.0, 1), (1.0, -6), (0.9921875, -7), (0.99219, -6), (254.0, 1),
                 (0.0, -50), (2.0 ** -60, -50), (1e30, 50), (np.inf, 50)):
        assert choose.grid([a, 0.0]) == 2.0 ** e, a
        assert choose.grid([0.0, -a]) == 2.0 ** e, a


def test_bounds_by_hand():
    hi, lo, s = choose.bounds([[1.0, -3.0, 0.0, 100.0], [2.5, -3.0, 0.0, -126.5]])
    assert s == 1.0
    assert hi.tolist() == [3, -3, 0, 100] and lo.tolist() == [1, -3, 0, -127]
    x, t = choose.query([0.5, -1.5, 2.5, 126.0])           # ties to even
    assert t == 1.0 and x.tolist() == [0, -2, 2, 126]
    # max(0*3, 0*1) + max(-2*-3, -2*-3) + 0 + max(126*100, 126*-127)
    assert choose.score([[0.5, -1.5, 2.5, 126.0]], (hi, lo, s)) == 6 + 12600


@pytest.mark.parametrize("d", [64, 128])
def test_score_bounds_every_product(d):
    """s hi and s lo enclose the keys, and the score is not below any product of
    the rounded query with a key of the page."""
    rng = np.random.default_rng(d)
    for trial in range(50):
        k = rng.normal(size=(rng.integers(1, 40), d)) * np.exp(rng.normal(size=d))
        hi, lo, s = choose.bounds(k)
        assert (k <= hi * s).all() and (k >= lo * s).all()
        assert max(abs(hi).max(), abs(lo).max()) <= 127
        q = rng.normal(size=d)
        x, t = choose.query(q)
        assert np.abs(x * t - q).max() <= t / 2
        assert choose.score([q], (hi, lo, s)) >= (k @ (x * t)).max() * (1 - 1e-12)
        assert abs(choose.score([q], (hi, lo, s)) / s / t) < 2 ** 21


def test_kept_pages():
    s = [9.0, 1.0, 5.0, 5.0, 5.0, 7.0, 0.0, 3.0]
    assert choose.kept(s, 8, 1, 1, 2) == [0, 2, 5, 7]       # a tie takes the lower page
    assert choose.kept(s, 8, 0, 1, 3) == [0, 2, 5, 7]
    assert choose.kept(s, 8, 0, 2, 0) == [6, 7]
    assert choose.kept(s, 8, 2, 2, 4) == list(range(8))
    assert choose.kept(s, 3, 1, 1, 5) == [0, 1, 2]
    assert choose.kept(s, 8, 3, 4, 0) == [0, 1, 2, 4, 5, 6, 7]


# ------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def lib():
    from head_aware_paged_gb300 import build
    build.build()
    from head_aware_paged_gb300 import _lib
    return _lib.load()


def test_null_handles(lib):
    from head_aware_paged_gb300._lib import i32_buffer
    one = i32_buffer([0, 1])
    at = one.buffer_info()[0]
    assert lib.sp_attach_page_bounds(None, None) == 1
    assert lib.sp_attention_decode_select(None, 0, at, 1, 256, 4, 1, 1, 0.0, 256, None, None, None) == 1
    assert lib.sp_append_kv_rope_axes(None, 0, at, 1, at, None, None, 0, None, 0, None, 0, None, None, 0, 0, 1, at, 1e4,
                                      None, None) == 1


def test_page_bounds_bytes(lib):
    from head_aware_paged_gb300 import Config, SegPagedError, sp_page_bounds_bytes
    cfg = dict(num_layers=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=64, max_seqs=4, max_seq_len=4096,
               num_pages=512, max_idx_per_seq=256, max_tokens=4096, max_batch=4)
    n = sp_page_bounds_bytes(Config(**cfg))
    assert n >= 512 * (256 + 4) + 2 * 8 * 65 * 4 + 8 * 4 and n <= 512 * 260 + 2 * 8 * 65 * 4 + 8 * 4 + 5 * 256
    with pytest.raises(SegPagedError):
        sp_page_bounds_bytes(Config(**dict(cfg, head_dim=96)))
    c = Config(**cfg).to_c()
    assert lib.sp_page_bounds_bytes(ctypes.byref(c), None) == 1


def test_rope_axes_refusals(lib):
    """Every refusal comes before the launch: addresses that are never read."""
    from head_aware_paged_gb300._lib import i32_buffer
    A = 1 << 20
    good = dict(q=A, qs=1024, hq=8, k=2 * A, ks=256, hkv=2, d=128, rows=4, pos=3 * A, ax=4, rs=1, n=3,
                of=[0] * 32 + [1] * 16 + [2] * 16, theta=1e4, fr=None, qo=4 * A, ko=5 * A)

    def call(**kw):
        a = dict(good, **kw)
        of = None if a["of"] is None else i32_buffer(a["of"])
        fr = None if a["fr"] is None else (ctypes.c_double * len(a["fr"]))(*a["fr"])
        return lib.sp_rope_axes(a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["hkv"], a["d"], a["rows"], a["pos"], a["ax"],
                                a["rs"], a["n"], of and of.buffer_info()[0], a["theta"], fr, a["qo"], a["ko"], None)

    assert call(rows=0) == 0 and call(hq=0, hkv=0) == 0 and call(rows=0, pos=None, q=None, k=None) == 0
    assert call(d=96) == 3
    bad = [dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(of=None), dict(n=0), dict(n=5),
           dict(of=[3] * 64), dict(of=[-1] * 64), dict(hq=-1), dict(hkv=2000), dict(rows=-1), dict(rows=1 << 31),
           dict(qs=1023), dict(qs=1028), dict(ks=255), dict(q=A + 8), dict(ko=5 * A + 2), dict(pos=3 * A + 4),
           dict(ax=-1), dict(rs=-1), dict(theta=0.0), dict(theta=float("nan")), dict(theta=float("inf")),
           dict(fr=[float("nan")] * 64), dict(fr=[1e6] * 64),
           dict(qo=2 * A), dict(qo=2 * A + 512), dict(qo=5 * A), dict(qo=5 * A + 1024), dict(ko=A), dict(ko=A + 2 * 1024 * 3),
           dict(qo=A, qs=1032), dict(qo=A + 2048), dict(ko=3 * A), dict(qo=3 * A + 96 - 16), dict(ko=4 * A + 16)]
    for kw in bad:
        assert call(**kw) == 1, kw
