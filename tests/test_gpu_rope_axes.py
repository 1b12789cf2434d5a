"""GPU: rotation by positions on several axes, rows to rows (sp_rope_axes) and on
the way into the pages (sp_append_kv_rope_axes).

Rotated values are compared with the closed form in 64 bits: half a bf16 step of
the value (2^-8) plus fp32 slack relative to the rotated pair (three roundings
and the cosine's and sine's own, 2^-21) and the angle's own error of |p w| 2^-53
radians.  What the two calls share is compared bit for bit."""
import numpy as np
import pytest
import torch

import workloads as W
from _gpu_common import f64, gpu_ready, to_c_policies

pytestmark = pytest.mark.gpu

G, L, R = W.GLOBAL, W.LOCAL, W.RETRIEVAL


def _mk(hq, hkv, d, P, seqs, max_len, pages, kv="bf16", batch=None):
    import head_aware_paged_gb300 as H
    return H.SegPagedCache(H.Config(num_layers=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P,
                                    max_seqs=seqs, max_seq_len=max_len, num_pages=pages, max_idx_per_seq=8192,
                                    max_tokens=max_len, max_batch=batch or seqs,
                                    kv_dtype={"bf16": H.KV_BF16, "fp8": H.KV_FP8, "fp4": H.KV_FP4}[kv]))


def _turned(x, pos, of, theta=10000.0, freq=None):
    """x [n, heads, d] (bf16) turned by pos [axes, n], 64 bits; with its tolerance."""
    x = f64(x)
    half = x.shape[-1] // 2
    w = np.asarray(freq if freq is not None else theta ** (-2.0 * np.arange(half) / (2 * half)), np.float64)
    a = np.asarray(pos, np.float64)[np.asarray(of)].T * w                    # [n, half]
    c, s = np.cos(np.fmod(a, 2 * np.pi))[:, None], np.sin(np.fmod(a, 2 * np.pi))[:, None]
    y = np.concatenate([x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s], -1)
    pair = np.hypot(x[..., :half], x[..., half:]) * (2.0 ** -21 + np.abs(a)[:, None] * 2.0 ** -52)
    return y, 2.0 ** -8 * np.abs(y) + np.concatenate([pair, pair], -1) + 1e-30


def _close(got, want, what):
    ref, tol = want
    assert tuple(got.shape) == ref.shape, what
    worst = (np.abs(f64(got) - ref) / tol).max() if ref.size else 0
    assert worst <= 1.0, "%s: %.3g of the tolerance" % (what, worst)


def _of(d, n, seed):
    return [int(x) for x in np.random.default_rng(seed).integers(0, n, d // 2)]


@pytest.mark.parametrize("n,hq,hkv,d,axes", [(1, 32, 8, 128, 3), (3, 14, 2, 64, 3), (777, 28, 4, 128, 3), (257, 1, 1, 64, 1),
                                             (2049, 5, 5, 128, 4), (5000, 35, 5, 64, 2), (64, 0, 8, 128, 3),
                                             (9, 16, 0, 64, 3), (5, 1024, 3, 64, 3)])
def test_rows_against_64_bits(n, hq, hkv, d, axes):
    import head_aware_paged_gb300 as H
    gpu_ready()
    x = W.normal((n, hq + 2 * hkv, d), n + hq, device="cuda")               # a fused projection's rows
    q, k = (x[:, :hq] if hq else None), (x[:, hq:hq + hkv] if hkv else None)
    rng = np.random.default_rng(n)
    pos = rng.integers(0, 200000, (axes, n))
    p, of = torch.from_numpy(pos).cuda(), _of(d, axes, n)
    qo, ko = H.sp_rope_axes(q, k, p, of, rope_theta=500000.0)
    for got, src, name in ((qo, q, "q"), (ko, k, "k")):
        assert (got is None) == (src is None)
        if got is not None:
            assert got.is_contiguous()
            _close(got, _turned(src, pos, of, 500000.0), name)
    # other layouts of the same positions give the same bits
    wide = torch.zeros(n, axes + 2, dtype=torch.int64, device="cuda")
    wide[:, 1:axes + 1] = p.T
    again = H.sp_rope_axes(q, k, wide.T[1:axes + 1], of, rope_theta=500000.0)
    for a, b in zip((qo, ko), again):
        assert a is None or torch.equal(a, b)


def test_far_negative_and_shared_positions():
    import head_aware_paged_gb300 as H
    gpu_ready()
    n, d = 40, 128
    q = W.normal((n, 4, d), 5, device="cuda")
    of = _of(d, 3, 5)
    pos = np.stack([np.arange(n) * 100003 - 2000000, np.full(n, -1), np.arange(n) + (1 << 33)])
    qo, _ = H.sp_rope_axes(q, None, torch.from_numpy(pos).cuda(), of)
    _close(qo, _turned(q, pos, of), "far")
    # positions near 2^62: whole turns away from small ones
    freq = [2 * np.pi / 8.0] * 64                                            # an eighth of a turn a position
    big = torch.tensor([[(1 << 62) + 8 * i + i % 8 for i in range(n)]], device="cuda")
    small = torch.tensor([[i % 8 for i in range(n)]], device="cuda")
    a = H.sp_rope_axes(q, None, small, [0] * 64, inv_freq=freq)[0]
    assert torch.equal(a, H.sp_rope_axes(q, None, big, [0] * 64, inv_freq=freq)[0])
    # one position that all rows share (stride 0)
    one = torch.tensor([[7], [9]], device="cuda")
    of2 = _of(d, 2, 6)
    a = H.sp_rope_axes(q, None, one.expand(2, n), of2)[0]
    assert torch.equal(a, H.sp_rope_axes(q, None, one.repeat(1, n), of2)[0])


def test_zero_positions_and_in_place():
    import head_aware_paged_gb300 as H
    gpu_ready()
    q, k = W.normal((33, 6, 64), 1, device="cuda"), W.normal((33, 2, 64), 2, device="cuda")
    zero = torch.zeros(3, 33, dtype=torch.int64, device="cuda")
    qo, ko = H.sp_rope_axes(q, k, zero, _of(64, 3, 1))
    assert torch.equal(qo, q) and torch.equal(ko, k)
    p = torch.randint(0, 9999, (3, 33), device="cuda")
    qo, ko = H.sp_rope_axes(q, k, p, _of(64, 3, 1))
    q2, k2 = q.clone(), k.clone()
    got = H.sp_rope_axes(q2, k2, p, _of(64, 3, 1), q_out=q2, k_out=k2)
    assert got[0] is q2 and torch.equal(q2, qo) and torch.equal(k2, ko)
    with pytest.raises(AssertionError):
        H.sp_rope_axes(q, k, p.int(), _of(64, 3, 1))
    with pytest.raises(H.SegPagedError):
        H.sp_rope_axes(q, k, p, [3] * 32)
    with pytest.raises(AssertionError):
        H.sp_rope_axes(q, k, p[:, :32], _of(64, 3, 1))


def test_another_stream():
    import head_aware_paged_gb300 as H
    gpu_ready()
    q = W.normal((4096, 8, 128), 1, device="cuda")
    p = torch.randint(0, 9999, (3, 4096), device="cuda")
    want = H.sp_rope_axes(q, None, p, _of(128, 3, 1))[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = H.sp_rope_axes(q, None, p, _of(128, 3, 1))[0]
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kv,d,P,hq,hkv", [("bf16", 64, 16, 6, 2), ("bf16", 128, 64, 32, 8), ("fp8", 128, 32, 8, 2),
                                           ("fp4", 128, 64, 16, 4), ("fp4", 128, 16, 3, 1)])
def test_equal_axes_are_the_token_positions(kv, d, P, hq, hkv):
    """Positions that say where the tokens are stored: append_kv_rope, bit for
    bit, in pages, tables and queries (ragged calls, overwrites included)."""
    gpu_ready()
    tot = 500
    pol = [[W.HeadPolicy(G), W.HeadPolicy(L, 5, 70), W.HeadPolicy(R, idx=np.arange(1, tot, 3, dtype=np.int32)),
            W.HeadPolicy(L, 0, 1), W.HeadPolicy(G), W.HeadPolicy(L, 40, 300), W.HeadPolicy(G), W.HeadPolicy(G)][:hkv]]
    a, b = (_mk(hq, hkv, d, P, 3, tot, 3 * hkv * (tot // P + 4), kv) for _ in range(2))
    rng = np.random.default_rng(P)
    ks = np.exp2(rng.integers(-3, 3, (hkv, d))).astype(np.float32)
    for c in (a, b):
        if kv != "bf16":
            c.set_kv_scales(0, ks, ks)
        for s in range(3):
            c.set_policy(s, to_c_policies(pol))
    n = [0, 0, 0]
    for call in range(6):
        new = [int(rng.integers(0, 90)) for _ in range(3)] if call else [1, 0, 77]
        at = [x - min(x, 20) if call == 4 else x for x in n]
        cu = [0, new[0], new[0] + new[1], sum(new)]
        if not cu[-1]:
            continue
        x = W.normal((cu[-1], hq + 2 * hkv, d), call, device="cuda")
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        tok = torch.cat([torch.arange(i, i + c) for i, c in zip(at, new)]).cuda()
        qa = a.append_kv_rope(0, [2, 0, 1], cu, q, k, v, pos=at, rope_theta=500000.0)
        qb = b.append_kv_rope_axes(0, [2, 0, 1], cu, q, k, v, tok.expand(3, -1), _of(d, 3, call), pos=at,
                                   rope_theta=500000.0)
        assert torch.equal(qa, qb)
        n = [max(o, i + c) for o, i, c in zip(n, at, new)]
    assert torch.equal(a.pool, b.pool) and torch.equal(a.meta[:-256], b.meta[:-256]) and a.status() == 0 and b.status() == 0


@pytest.mark.parametrize("n,d,hq,hkv", [(1, 128, 32, 8), (200, 64, 14, 2), (700, 128, 12, 4)])
def test_append_is_rotation_then_append(n, d, hq, hkv):
    """On bf16 pages: the rotated rows of sp_rope_axes, stored by append_kv."""
    import head_aware_paged_gb300 as H
    gpu_ready()
    a, b = (_mk(hq, hkv, d, 64, 2, 800, 2 * hkv * 14) for _ in range(2))
    pol = [[W.HeadPolicy(G) if h % 2 == 0 else W.HeadPolicy(L, 4, 100) for h in range(hkv)]]
    for c in (a, b):
        for s in range(2):
            c.set_policy(s, to_c_policies(pol))
    x = W.normal((n + 3, hq + 2 * hkv, d), n, device="cuda")
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    pos = torch.randint(-5, 100000, (3, n + 3), device="cuda")
    of = _of(d, 3, n)
    cu = [0, n, n + 3]
    qa = a.append_kv_rope_axes(0, [0, 1], cu, q, k, v, pos, of)
    qb, kb = H.sp_rope_axes(q, k, pos, of)
    b.append_kv(0, [0, 1], cu, kb, v.contiguous())
    assert torch.equal(qa, qb) and torch.equal(a.pool, b.pool)
    _close(qa, _turned(q, pos.cpu().numpy(), of), "q")
    # keys alone
    for c in (a, b):
        c.release(0)
    assert a.append_kv_rope_axes(0, [0], [0, n], None, k[:n], v[:n], pos, of) is None
    b.append_kv(0, [0], [0, n], kb[:n].contiguous(), v[:n].contiguous())
    assert torch.equal(a.pool, b.pool)


def test_replay_reads_the_positions_then():
    gpu_ready()
    hq, hkv, d = 8, 2, 128
    c = _mk(hq, hkv, d, 64, 2, 300, 64)
    for s in range(2):
        c.set_policy(s, to_c_policies([[W.HeadPolicy(G), W.HeadPolicy(L, 4, 100)]]))
        k = W.normal((100, hkv, d), s, device="cuda")
        c.build(s, 0, k, k)
    x = W.normal((2, hq + 2 * hkv, d), 9, device="cuda")
    q, k, v = x[:, :hq].contiguous(), x[:, hq:hq + hkv].contiguous(), x[:, hq + hkv:].contiguous()
    pos = torch.zeros(3, 2, dtype=torch.int64, device="cuda")
    of = _of(d, 3, 2)
    args = (0, [0, 1], [0, 1, 2], q, k, v, pos, of)
    out = torch.empty_like(q)
    c.append_kv_rope_axes(*args, pos=[99, 99], q_out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append_kv_rope_axes(*args, pos=[99, 99], q_out=out)
    for r in range(3):
        pos.copy_(torch.randint(0, 5000, (3, 2), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        _close(out, _turned(q, pos.cpu().numpy(), of), "replay %d" % r)
        pool = c.pool.clone()
        eager = c.append_kv_rope_axes(*args, pos=[99, 99])
        assert torch.equal(eager, out) and torch.equal(c.pool, pool)
    assert c.status() == 0


def test_append_refusals():
    import head_aware_paged_gb300 as H
    gpu_ready()
    c = _mk(8, 2, 128, 64, 2, 300, 64)
    c.set_policy(0, to_c_policies([[W.HeadPolicy(G), W.HeadPolicy(G)]]))
    x = W.normal((4, 12, 128), 9, device="cuda")
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    pos = torch.zeros(3, 4, dtype=torch.int64, device="cuda")
    of = [0] * 64
    before = c.meta.clone()
    for bad in (dict(axis_of=[3] * 64), dict(axis_of=[-1] * 64), dict(axis_pos=torch.zeros(5, 4, dtype=torch.int64, device="cuda")),
                dict(rope_theta=-1.0), dict(pos=[1]), dict(inv_freq=[1e9] * 64)):
        a = dict(axis_pos=pos, axis_of=of)
        a.update(bad)
        with pytest.raises(H.SegPagedError):
            c.append_kv_rope_axes(0, [0], [0, 4], q, k, v, **a)
    buf = torch.zeros(3 * 4 * 8 + 4 * 8 * 128 * 2, dtype=torch.uint8, device="cuda")
    over = buf[:96].view(torch.int64).view(3, 4)
    with pytest.raises(H.SegPagedError):                                     # the queries' rows end inside the positions
        c.append_kv_rope_axes(0, [0], [0, 4], q, k, v, over, of, q_out=buf[64:64 + 8192].view(torch.bfloat16).view(4, 8, 128))
    for bad in (dict(axis_pos=pos.int()), dict(axis_pos=pos[:, :3]), dict(axis_of=[0] * 63), dict(axis_pos=pos.cpu())):
        a = dict(axis_pos=pos, axis_of=of)
        a.update(bad)
        with pytest.raises(AssertionError):
            c.append_kv_rope_axes(0, [0], [0, 4], q, k, v, **a)
    assert torch.equal(c.meta, before) and c.seq_len(0, 0) == 0
    c.append_kv_rope_axes(0, [0], [0, 0], q[:0], k[:0], v[:0], pos[:, :0], of)      # no rows: nothing to do
    assert c.seq_len(0, 0) == 0 and c.status() == 0
