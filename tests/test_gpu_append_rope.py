"""GPU: sp_append_kv_rope -- the rotary embedding of new queries and keys on
their way to the attention and into the pages.

Rotated values are compared with the closed form in 64 bits (oracle/rope.py):
half a bf16 step of the value (2^-8) plus fp32 slack relative to the rotated
pair (three roundings and the cosine's and sine's own, 2^-21).  Where rows go
is integer work: page tables and untouched bytes are compared exactly."""
import numpy as np
import pytest
import torch

import workloads as W
from _gpu_common import f64, gpu_ready, to_c_policies
from oracle import fp4, fp8, rope

pytestmark = pytest.mark.gpu

G, L, R = W.GLOBAL, W.LOCAL, W.RETRIEVAL


def _mk(hq, hkv, d, P, seqs, max_len, pages, kv="bf16", layers=1, batch=None):
    import head_aware_paged_gb300 as H
    return H.SegPagedCache(H.Config(num_layers=layers, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P,
                                    max_seqs=seqs, max_seq_len=max_len, num_pages=pages, max_idx_per_seq=8192,
                                    max_tokens=max_len, max_batch=batch or seqs,
                                    kv_dtype={"bf16": H.KV_BF16, "fp8": H.KV_FP8, "fp4": H.KV_FP4}[kv]))


def _turn(x, pos, theta=10000.0, freq=None):
    """x [n, heads, d] (bf16) turned to positions pos, 64 bits."""
    x = f64(x)
    half = x.shape[-1] // 2
    w = np.asarray(freq if freq is not None else theta ** (-2.0 * np.arange(half) / (2 * half)), np.float64)
    a = np.fmod(np.asarray(pos, np.float64)[:, None] * w, 2 * np.pi)[:, None]
    c, s = np.cos(a), np.sin(a)
    return np.concatenate([x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s], -1)


def _close(got, ref, what):
    assert tuple(got.shape) == ref.shape, what
    half = ref.shape[-1] // 2
    pair = np.hypot(ref[..., :half], ref[..., half:])
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * np.concatenate([pair, pair], -1) + 1e-30
    worst = (np.abs(f64(got) - ref) / tol).max() if ref.size else 0
    assert worst <= 1.0, "%s: %.3g of the tolerance" % (what, worst)


def _rows(cache, seq, h, layer=0):
    ids, pos = cache.export_table(seq, layer, h)
    r = [(p, pg, s) for pg, slots in zip(ids, pos) for s, p in enumerate(slots) if p >= 0]
    return [np.array(x, dtype=np.int64) for x in zip(*r)] if r else None


def _fused(n, hq, hkv, d, seed):
    """One projection's output: q, k, v are views of it, rows apart."""
    x = W.normal((n, hq + 2 * hkv, d), seed, device="cuda")
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


@pytest.mark.parametrize("kv,d,P,hq,hkv", [("bf16", 64, 16, 6, 2), ("bf16", 128, 64, 32, 8), ("bf16", 128, 128, 5, 5),
                                           ("fp8", 128, 32, 8, 2), ("fp4", 128, 64, 16, 4), ("fp4", 128, 16, 3, 1)])
def test_matches_append_and_the_rotation(kv, d, P, hq, hkv):
    """Ragged appends in several calls: the page tables are those of
    append_kv, the stored keys the rotated ones, the values as they came."""
    gpu_ready()
    rng = np.random.default_rng(P + hq)
    tot = 700
    pol = [[W.HeadPolicy(G), W.HeadPolicy(L, 5, 70), W.HeadPolicy(R, idx=np.arange(1, tot, 3, dtype=np.int32)),
            W.HeadPolicy(L, 0, 1), W.HeadPolicy(R, idx=np.zeros(0, np.int32)), W.HeadPolicy(L, 40, 300),
            W.HeadPolicy(G), W.HeadPolicy(G)][:hkv]]
    a, b = (_mk(hq, hkv, d, P, 3, tot, 3 * hkv * (tot // P + 4), kv) for _ in range(2))
    ks = np.exp2(rng.integers(-3, 3, (hkv, d))).astype(np.float32)
    for c in (a, b):
        if kv == "fp8":
            c.set_kv_scales(0, ks, ks)
        for s in range(3):
            c.set_policy(s, to_c_policies(pol))
    data = [_fused(tot, hq, hkv, d, 70 + s) for s in range(3)]
    n = [0, 0, 0]
    for call in range(5):
        seqs = [[0, 1, 2], [2, 0], [1], [0, 1, 2], [1, 2]][call]
        cnt = [int(rng.choice([0, 1, 2, 17, 130])) for _ in seqs]
        cu = [0] + list(np.cumsum(cnt))
        part = [torch.cat([data[s][i][n[s]:n[s] + c] for s, c in zip(seqs, cnt)]) for i in range(3)]
        wide = torch.empty(max(1, cu[-1]), hq + 2 * hkv + 1, d, dtype=torch.bfloat16, device="cuda")
        q, k, v = wide[:cu[-1], :hq], wide[:cu[-1], hq:hq + hkv], wide[:cu[-1], hq + hkv:hq + 2 * hkv]
        for x, y in zip((q, k, v), part):
            x.copy_(y)
        got = a.append_kv_rope(0, seqs, cu, q, k, v)
        if cu[-1]:
            b.append_kv(0, seqs, cu, part[1].contiguous(), part[2].contiguous())
        pos = np.concatenate([np.arange(n[s], n[s] + c) for s, c in zip(seqs, cnt)] + [np.zeros(0)])
        _close(got, _turn(part[0], pos), "queries")
        for s, c in zip(seqs, cnt):
            n[s] += c
            assert a.seq_len(s, 0) == n[s] == b.seq_len(s, 0)
    assert a.free_pages() == b.free_pages()
    for s in range(3):
        for h in range(hkv):
            assert a.export_table(s, 0, h) == b.export_table(s, 0, h)
            r = _rows(a, s, h)
            if r is None:
                continue
            p, pg, sl = r
            ref = _turn(data[s][1], np.arange(tot))[p, h]
            if kv == "bf16":
                _close(a.k_pool()[pg, sl], ref, "keys")
                assert torch.equal(a.v_pool()[pg, sl], data[s][2][torch.tensor(p).cuda(), h])
            elif kv == "fp8":
                got, raw = fp8.decode(a.k_pool()[pg, sl].cpu().numpy()), ref / ks[h]
                step = np.exp2(np.floor(np.log2(np.maximum(np.abs(raw), 2.0 ** -6))) - 3)
                assert (np.abs(got - raw) <= step / 2 * 1.001 + 2.0 ** -20).all()
                assert torch.equal(a.v_pool()[pg, sl], b.v_pool()[pg, sl])
            else:
                kp, vp, vb = (x.cpu().numpy() for x in (a.k_pool(), a.v_pool(), b.v_pool()))
                for i in range(len(p)):
                    code, sc = fp4.read_row(kp[pg[i], sl[i] // 16], sl[i] % 16, False)
                    scl = np.repeat(fp4.SCALES[sc], 16)
                    top = np.abs(ref[i]).reshape(8, 16).max(1) / 6
                    assert (np.abs(fp4.SCALES[sc] / top - 1) <= 2.0 ** -4 + 1e-5).all()
                    y = np.abs(ref[i]) / scl
                    half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0)) * scl
                    err = np.abs(fp4.dequantize(code, sc) - ref[i])
                    assert (err <= half * 1.001 + 0.07 * np.abs(ref[i]) * (y > 5.9)).all()
                assert (vp == vb).all()
    assert a.status() == 0


@pytest.mark.parametrize("theta,freq", [(10000.0, None), (500000.0, None), (1.0, "own")])
def test_far_positions(theta, freq):
    """Position 131,071 of a sequence whose heads keep 64 tokens, next to the
    first ones; own frequencies, among them 0 (no rotation) and negative ones."""
    gpu_ready()
    hq, hkv, d, P, n = 4, 2, 128, 64, 131000
    cache = _mk(hq, hkv, d, P, 2, 131072, 64)
    f = None
    if freq:
        f = np.linspace(-1.0, 2.0, d // 2)
        f[5], f[6] = 0.0, 65536.0
    for s in range(2):
        cache.set_policy(s, to_c_policies([[W.HeadPolicy(L, 4, 64)] * hkv]))
    old = W.normal((n, hkv, d), 1, device="cuda")
    cache.build(0, 0, old, old)
    q, k, v = _fused(72 + 3, hq, hkv, d, 2)
    got = cache.append_kv_rope(0, [0, 1], [0, 72, 75], q, k, v, rope_theta=theta, inv_freq=f)
    pos = np.concatenate([np.arange(n, n + 72), np.arange(3)])
    _close(got, _turn(q, pos, theta, f), "queries")
    for s, (lo, cnt) in enumerate(((n, 72), (0, 3))):
        p, pg, sl = _rows(cache, s, 1)
        new = p >= lo
        want = _turn(k, pos, theta, f)[(0 if s == 0 else 72) + p[new] - lo, 1]
        _close(cache.k_pool()[pg[new], sl[new]], want, "keys")
        if s == 0:                                       # older rows are as they were
            old_p = torch.tensor(p[~new]).cuda()
            assert torch.equal(cache.k_pool()[pg[~new], sl[~new]], old[old_p, 1])
    if f is not None:
        assert torch.equal(got[:, :, 5], q[:, :, 5]) and torch.equal(got[:, :, 5 + d // 2], q[:, :, 5 + d // 2])
    assert cache.status() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_overwriting_held_positions(kv):
    """pos inside what is held: those rows are rewritten where the head keeps
    them, the rest is appended, everything else keeps its bytes."""
    gpu_ready()
    hq, hkv, d, P, n = 6, 3, 128, 16, 200
    cache = _mk(hq, hkv, d, P, 2, 400, 2 * hkv * 30, kv)
    pols = [[W.HeadPolicy(G), W.HeadPolicy(L, 5, 40), W.HeadPolicy(R, idx=np.arange(0, 400, 7, dtype=np.int32))]]
    for s in range(2):
        cache.set_policy(s, to_c_policies(pols))
        cache.build(s, 0, W.normal((n, hkv, d), s, device="cuda"), W.normal((n, hkv, d), s + 5, device="cuda"))
    tables = [cache.export_table(1, 0, h) for h in range(hkv)]
    start, cnt = [0, 190], [10, 30]
    q, k, v = _fused(40, hq, hkv, d, 9)
    kp0, vp0 = cache.k_pool().clone(), cache.v_pool().clone()
    got = cache.append_kv_rope(0, [0, 1], [0, 10, 40], q, k, v, pos=start)
    assert [cache.seq_len(s, 0) for s in range(2)] == [200, 220]
    pos = np.concatenate([np.arange(a, a + c) for a, c in zip(start, cnt)])
    _close(got, _turn(q, pos), "queries")
    same = torch.ones(cache.k_pool().shape[:2], dtype=torch.bool, device="cuda")
    for s in range(2):
        for h in range(hkv):
            r = _rows(cache, s, h)
            p, pg, sl = r
            new = (p >= start[s]) & (p < start[s] + cnt[s])
            at = np.array([(0 if s == 0 else 10) + x - start[s] for x in p[new]], dtype=np.int64)
            if kv == "bf16":
                if len(at):
                    _close(cache.k_pool()[pg[new], sl[new]], _turn(k, pos)[at, h], "keys")
                    assert torch.equal(cache.v_pool()[pg[new], sl[new]], v[torch.tensor(at).cuda(), h])
                same[pg[new], sl[new]] = False
            else:
                vp = cache.v_pool().cpu().numpy()
                for i, t in zip(np.nonzero(new)[0], at):
                    code, sc = fp4.read_row(vp[pg[i], sl[i] // 16], sl[i] % 16, True)
                    want = fp4.quantize(f64(v[t, h]))
                    assert (sc == want[1]).all()
                    assert ((code == want[0]) | ((code & 7 == 0) & (want[0] & 7 == 0))).all()
                    same[pg[i], sl[i] // 16] = False
    assert torch.equal(cache.k_pool()[same], kp0[same]) and torch.equal(cache.v_pool()[same], vp0[same])
    for h in range(hkv):                                 # pages held before stay where they were
        assert cache.export_table(1, 0, h)[0][:len(tables[h][0])] == tables[h][0]
    # the same call again changes nothing
    kp1 = cache.k_pool().clone()
    cache.append_kv_rope(0, [0, 1], [0, 10, 40], q, k, v, pos=start)
    assert torch.equal(cache.k_pool(), kp1) and cache.seq_len(1, 0) == 220
    assert cache.status() == 0


def test_many_sequences_keys_only_and_in_place():
    """More sequences than the small parameter record holds; no queries; the
    queries rotated in place; another layer and stream."""
    gpu_ready()
    hq, hkv, d, P, B = 16, 8, 64, 16, 130
    cache = _mk(hq, hkv, d, P, B, 400, B * hkv * 4, layers=2)
    for s in range(B):
        cache.set_policy(s, to_c_policies([[W.HeadPolicy(G)] * hkv] * 2))
    cnt = [1 + (7 * s) % 5 for s in range(B)]
    cu = [0] + [int(x) for x in np.cumsum(cnt)]
    q, k, v = _fused(cu[-1], hq, hkv, d, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert cache.append_kv_rope(1, list(range(B)), cu, None, k, v) is None
        x = q.contiguous().clone()
        y = cache.append_kv_rope(1, list(range(B)), cu, x, k, v, pos=[0] * B, q_out=x)
    side.synchronize()
    assert y is x
    pos = np.concatenate([np.arange(c) for c in cnt])
    _close(x, _turn(q, pos), "queries in place")
    ref = _turn(k, pos)
    for s in (0, 31, 32, 77, B - 1):
        assert cache.seq_len(s, 1) == cnt[s] and cache.seq_len(s, 0) == 0
        p, pg, sl = _rows(cache, s, 7, layer=1)
        _close(cache.k_pool()[pg, sl], ref[cu[s] + p, 7], "keys")
    assert cache.free_pages() == B * hkv * 4 - B * hkv
    assert cache.status() == 0


def test_release_then_append_and_graph_replay():
    gpu_ready()
    hq, hkv, d, P = 4, 2, 64, 16
    cache = _mk(hq, hkv, d, P, 2, 128, 40)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G), W.HeadPolicy(L, 4, 20)]]))
    q, k, v = _fused(60, hq, hkv, d, 4)
    cache.append_kv_rope(0, [0], [0, 60], q, k, v)
    cache.release(0)
    assert cache.free_pages() == 40
    cache.append_kv_rope(0, [0], [0, 50], q, k, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = cache.append_kv_rope(0, [0], [0, 10], q[50:], k[50:], v[50:])
    assert cache.seq_len(0, 0) == 60                     # the call counts when it is captured
    for _ in range(2):                                   # a replay writes the same positions and pages again
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _close(got, _turn(q[50:], np.arange(50, 60)), "replayed")
        p, pg, sl = _rows(cache, 0, 0)
        assert p.tolist() == list(range(60))
        _close(cache.k_pool()[pg, sl], _turn(k, np.arange(60))[p, 0], "keys")
    assert cache.status() == 0


def test_refusals_change_nothing():
    gpu_ready()
    from head_aware_paged_gb300 import SegPagedError, sp_append_kv_rope
    hq, hkv, d = 4, 2, 64
    cache = _mk(hq, hkv, d, 16, 2, 100, 12, batch=2)
    for s in range(2):
        cache.set_policy(s, to_c_policies([[W.HeadPolicy(G)] * hkv]))
    q, k, v = _fused(60, hq, hkv, d, 4)
    cache.append_kv_rope(0, [0], [0, 10], q, k, v)
    before = cache.k_pool().clone()
    kc = k.contiguous()
    cases = [dict(seqs=[0, 0]), dict(seqs=[2]), dict(layer=1), dict(cu=[0, 101]), dict(cu=[1, 5]), dict(cu=[0, 5, 4], seqs=[0, 1]),
             dict(pos=[11]), dict(pos=[-1]), dict(theta=0.0), dict(theta=float("nan")), dict(freq=[1e9] * 32),
             dict(freq=[float("nan")] * 32), dict(cu=[0, 95]), dict(cu=[0, 60], seqs=[1], pages=True)]
    for c in cases:
        cu = c.get("cu", [0, 4])
        seqs = c.get("seqs", [0])
        if c.get("pages"):                               # 8 more pages are needed, fewer are free
            cache.append_kv_rope(0, [0], [0, 59], q, k, v)
            before = cache.k_pool().clone()
        n0, free = cache.seq_len(0, 0), cache.free_pages()
        with pytest.raises(SegPagedError):
            sp_append_kv_rope(cache.handle, c.get("layer", 0), seqs, cu, q, k, v, torch.empty_like(q),
                              pos=c.get("pos"), rope_theta=c.get("theta", 1e4), inv_freq=c.get("freq"))
        assert cache.seq_len(0, 0) == n0 and cache.free_pages() == free
    for args in ((None, torch.empty_like(q)), (q, None)):
        with pytest.raises(SegPagedError):
            sp_append_kv_rope(cache.handle, 0, [0], [0, 4], args[0], k, v, args[1])
    flat = W.normal((8 * hkv * d + 8,), 1, device="cuda")
    bad = flat[1:1 + 4 * hkv * d].view(4, hkv, d)        # not 16-byte aligned
    with pytest.raises(SegPagedError):
        sp_append_kv_rope(cache.handle, 0, [0], [0, 4], None, bad, kc[:4], None)
    with pytest.raises(SegPagedError):                   # row stride not a multiple of 8
        sp_append_kv_rope(cache.handle, 0, [0], [0, 4], None, flat.as_strided((4, hkv, d), (hkv * d + 1, d, 1)), kc[:4], None)
    for bad_args in (dict(k=k.float()), dict(k=k[:, :1]), dict(cu=[0, 61]), dict(pos=[0, 0]), dict(freq=[0.1])):
        with pytest.raises(AssertionError):
            cache.append_kv_rope(0, [0], bad_args.get("cu", [0, 4]), q, bad_args.get("k", k), v,
                                 pos=bad_args.get("pos"), inv_freq=bad_args.get("freq"))
    assert torch.equal(cache.k_pool(), before)
    assert cache.append_kv_rope(0, [0], [0, 0], q[:0], k[:0], v[:0]).shape == (0, hq, d)
    assert cache.status() == 0


def test_captured_call_that_needs_pages_is_refused():
    """Pages are taken from the free stack when the kernel runs; a replay would
    take whatever lies there by then.  The refused call changes nothing."""
    gpu_ready()
    from head_aware_paged_gb300 import SegPagedError
    hq, hkv, d, P = 4, 2, 64, 16
    cache = _mk(hq, hkv, d, P, 2, 128, 40)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G), W.HeadPolicy(L, 4, 20)]]))
    q, k, v = _fused(80, hq, hkv, d, 4)
    cache.append_kv_rope(0, [0], [0, 50], q, k, v)
    free, before = cache.free_pages(), cache.k_pool().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        with pytest.raises(SegPagedError) as e:
            cache.append_kv_rope(0, [0], [0, 20], q[50:], k[50:], v[50:])      # 50 + 20 tokens: a fifth page
        q[:1].clone()
    assert e.value.status == 3
    assert cache.seq_len(0, 0) == 50 and cache.free_pages() == free
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.k_pool(), before)
    cache.append_kv_rope(0, [0], [0, 20], q[50:], k[50:], v[50:])
    assert cache.seq_len(0, 0) == 70 and cache.free_pages() == free - 1
    assert cache.status() == 0


def test_replay_after_other_sequences_and_its_own_moved_on():
    """Between replays other sequences take and release pages and the written one
    grows past its ring: a replay still writes only its positions that are held,
    and leaves lengths, tables and every other row alone.  After a release of
    its sequence it writes nothing and says so."""
    gpu_ready()
    from head_aware_paged_gb300 import SegPagedError
    hq, hkv, d, P = 4, 3, 64, 16
    cache = _mk(hq * 3, hkv, d, P, 3, 256, 80)
    pol = [[W.HeadPolicy(G), W.HeadPolicy(L, 4, 20), W.HeadPolicy(R, idx=np.arange(0, 256, 3, dtype=np.int32))]]
    for s in range(3):
        cache.set_policy(s, to_c_policies(pol))
    q, k, v = _fused(200, hq * 3, hkv, d, 4)
    cache.append_kv_rope(0, [0, 1], [0, 50, 120], q, k, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = cache.append_kv_rope(0, [0], [0, 10], q[50:60], k[50:60], v[50:60])
    graph.replay()
    torch.cuda.synchronize()
    for grow in (30, 60):                       # to 90 tokens (50 .. 59 still in the ring), to 150 (behind it)
        cache.release(1)
        cache.append_kv_rope(0, [2, 0], [0, 40, 40 + grow], q, k, v)
        cache.append_kv_rope(0, [1], [0, 33], q, k, v)
        n = cache.seq_len(0, 0)
        pools = cache.k_pool().clone(), cache.v_pool().clone()
        tables = [cache.export_table(b, 0, h) for b in range(3) for h in range(hkv)]
        free = cache.free_pages()
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _close(got, _turn(q[50:60], 50 + np.arange(10)), "replayed")
        assert torch.equal(cache.k_pool(), pools[0]) and torch.equal(cache.v_pool(), pools[1])
        assert tables == [cache.export_table(b, 0, h) for b in range(3) for h in range(hkv)]
        assert cache.free_pages() == free and cache.seq_len(0, 0) == n
    assert cache.status() == 0
    cache.release(0)
    cache.append_kv_rope(0, [1], [0, 60], q, k, v)          # takes the pages that were sequence 0's
    pools = cache.k_pool().clone(), cache.v_pool().clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.k_pool(), pools[0]) and torch.equal(cache.v_pool(), pools[1])
    with pytest.raises(SegPagedError) as e:
        cache.status()
    assert e.value.status == 5
    assert cache.status() == 0 and cache.export_table(0, 0, 0) == ([], [])


def test_q_out_may_not_overlap_what_is_read():
    """q_out may be q itself where q is contiguous; any other overlap with the
    inputs would be a race and is refused."""
    gpu_ready()
    from head_aware_paged_gb300 import SegPagedError
    hq, hkv, d, n = 4, 2, 64, 10
    cache = _mk(hq, hkv, d, 16, 1, 128, 20)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)] * hkv]))
    flat = W.normal((n * (hq + 2 * hkv) * d,), 1, device="cuda")
    x = flat.view(n, hq + 2 * hkv, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    before = flat.clone()
    size = n * hq * d
    for q_in, off in ((q, 0), (q, 3 * d), (q, flat.numel() - size), (flat[:size].view(n, hq, d), d)):
        with pytest.raises(SegPagedError) as e:
            cache.append_kv_rope(0, [0], [0, n], q_in, k, v, q_out=flat[off:off + size].view(n, hq, d))
        assert e.value.status == 1 and cache.seq_len(0, 0) == 0
    assert torch.equal(flat, before)
    own = q.contiguous()
    got = cache.append_kv_rope(0, [0], [0, n], own, k, v, q_out=own)
    _close(got, _turn(q, np.arange(n)), "in place")
    big = torch.empty(2 * size, dtype=torch.bfloat16, device="cuda")         # side by side: no overlap
    big[:size] = q.reshape(-1)
    got = cache.append_kv_rope(0, [0], [0, n], big[:size].view(n, hq, d), k, v, q_out=big[size:].view(n, hq, d))
    _close(got, _turn(q, np.arange(n, 2 * n)), "side by side")
    assert cache.status() == 0


def test_strides_of_single_rows_and_single_heads():
    """A dimension of one element may have any stride: one token taken out of a
    heads-first layout, one KV head out of a sequence-first one."""
    gpu_ready()
    hq, hkv, d, n = 4, 2, 64, 9
    cache = _mk(hq, hkv, d, 16, 1, 64, 8)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)] * hkv]))
    q, k, v = (W.normal((h, 1, d), h, device="cuda").transpose(0, 1) for h in (hq, hkv, hkv))
    assert q.stride(0) == d and q.shape == (1, hq, d)
    got = cache.append_kv_rope(0, [0], [0, 1], q, k, v)
    assert torch.equal(got, q)                                   # position 0
    got = cache.append_kv_rope(0, [0], [0, 1], q, k, v)
    _close(got, _turn(q, [1]), "one token")
    p, pg, sl = _rows(cache, 0, 1)
    _close(cache.k_pool()[pg, sl], _turn(torch.cat([k, k]), [0, 1])[:, 1], "keys")
    one = _mk(1, 1, d, 16, 1, 64, 8)
    one.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    q, k, v = (W.normal((1, n, d), 5 + i, device="cuda").transpose(0, 1) for i in range(3))
    assert k.stride(1) == n * d and k.shape == (n, 1, d)
    got = one.append_kv_rope(0, [0], [0, n], q, k, v)
    _close(got, _turn(q, np.arange(n)), "one head")
    p, pg, sl = _rows(one, 0, 0)
    _close(one.k_pool()[pg, sl], _turn(k, np.arange(n))[:, 0], "keys of one head")
    assert torch.equal(one.v_pool()[pg, sl], v[:, 0])
    assert cache.status() == 0 and one.status() == 0


def test_tensors_elsewhere_are_refused():
    """Host memory is not read or written by a kernel."""
    gpu_ready()
    hq, hkv, d = 4, 2, 64
    cache = _mk(hq, hkv, d, 16, 1, 64, 8)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)] * hkv]))
    q, k, v = (W.normal((3, h, d), h, device="cuda") for h in (hq, hkv, hkv))
    for bad in (dict(q=q.cpu()), dict(k=k.cpu()), dict(v=v.cpu()), dict(q_out=torch.empty_like(q, device="cpu"))):
        with pytest.raises(AssertionError):
            cache.append_kv_rope(0, [0], [0, 3], bad.get("q", q), bad.get("k", k), bad.get("v", v), q_out=bad.get("q_out"))
    assert cache.seq_len(0, 0) == 0 and cache.status() == 0
