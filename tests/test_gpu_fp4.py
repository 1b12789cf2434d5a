"""GPU: 4-bit K/V pages (SP_KV_FP4_E2M1).

Writes are integer work: every stored code and scale equals the plain
definition's (oracle/fp4.py) for the row at that slot.  Attention is compared
with 64-bit attention over the dequantised rows, with tolerances counted from
the kernels' roundings: decode rounds P to f16 (2^-11 of each weight) and,
with channel scales, the scaled query (2^-11 of each product); prefill rounds
P (2^-8) and, with channel scales, K and V rows (2^-8) to bf16."""
import numpy as np
import pytest
import torch

import workloads as W
from _attn64 import attend, check
from _gpu_common import f64, gpu_ready, pol_tuple, to_c_policies
from oracle import fp4, rope

pytestmark = pytest.mark.gpu

G, L, R = W.GLOBAL, W.LOCAL, W.RETRIEVAL
D = 128


def _mk(hq, hkv, P, seqs, max_len, pages, layers=1, max_idx=8192, batch=None):
    from head_aware_paged_gb300 import KV_FP4, Config, SegPagedCache
    return SegPagedCache(Config(num_layers=layers, num_q_heads=hq, num_kv_heads=hkv, head_dim=D,
                                page_size=P, max_seqs=seqs, max_seq_len=max_len, num_pages=pages,
                                max_idx_per_seq=max_idx, max_tokens=max_len, max_batch=batch or seqs,
                                kv_dtype=KV_FP4))


def _kv(n, hkv, seed, scale=1.0):
    k = W.normal((n, hkv, D), W.tensor_seed(seed, "k"), 0.5, device="cuda")
    v = W.normal((n, hkv, D), W.tensor_seed(seed, "v"), scale, device="cuda")
    strong = torch.ones(D, device="cuda")
    strong[torch.arange(5, D, 37)] = 9.0
    return (k.float() * strong).to(torch.bfloat16), v


def _held(cache, seq, layer, h):
    """{position: (K codes, K scales, V codes, V scales)} of a unit's slots."""
    ids, pos = cache.export_table(seq, layer, h)
    kp, vp = cache.k_pool().cpu().numpy(), cache.v_pool().cpu().numpy()
    out = {}
    for pg, slots in zip(ids, pos):
        for s, p in enumerate(slots):
            if p >= 0:
                out[p] = fp4.read_row(kp[pg, s // 16], s % 16, False) + fp4.read_row(vp[pg, s // 16], s % 16, True)
    return out


def _check_codes(cache, seq, layer, h, k, v, ks=None, vs=None, what=""):
    held = _held(cache, seq, layer, h)
    p = sorted(held)
    if not p:
        return 0
    for x, at, s in ((k, 0, ks), (v, 2, vs)):
        code, sc = fp4.quantize(f64(x[:, h])[p], None if s is None else s[h])
        np.testing.assert_array_equal(np.stack([held[i][at + 1] for i in p]), sc, err_msg=what)
        got = np.stack([held[i][at] for i in p])
        # a negative value that rounds to zero may carry either sign
        same = (got == code) | ((got & 7 == 0) & (code & 7 == 0))
        assert same.all(), what
    return len(p)


def _stored(x, s=None):
    """What rows x [n, hkv, d] are held as, in 64 bits on the device."""
    if x.shape[0] == 0:
        return x.double()
    xs = f64(x)
    out = np.stack([fp4.stored(xs[:, h], None if s is None else s[h]) for h in range(xs.shape[1])], 1)
    return torch.tensor(out, device="cuda")


def _policies(rng, hkv, n):
    row = []
    for h in range(hkv):
        kind = int(rng.integers(0, 3))
        if kind == G:
            row.append(W.HeadPolicy(G))
        elif kind == L:
            row.append(W.HeadPolicy(L, int(rng.integers(0, 40)), int(rng.integers(1, 700))))
        else:
            idx = np.sort(rng.choice(n + 50, int(rng.integers(0, min(n, 400) + 1)), replace=False))
            row.append(W.HeadPolicy(R, idx=idx.astype(np.int32)))
    return row


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("P,hq,hkv", [(64, 32, 8), (16, 8, 2), (128, 7, 1), (32, 24, 8), (64, 16, 1), (16, 48, 4)])
def test_codes_and_decode(P, hq, hkv, scaled):
    gpu_ready()
    rng = np.random.default_rng(P + hq)
    lens = [1, 2, 63, 64, 65, 2999, int(rng.integers(3, 2999))]
    B, max_len = len(lens), 3000
    cache = _mk(hq, hkv, P, B, max_len, B * hkv * (max_len // P + 4))
    ks = vs = None
    if scaled:
        ks = np.exp2(rng.uniform(-3, 3, (hkv, D))).astype(np.float32)
        vs = np.exp2(rng.uniform(-3, 3, (hkv, D))).astype(np.float32)
        cache.set_kv_scales(0, ks, vs)
    data, pols = [_kv(n, hkv, 10 + b) for b, n in enumerate(lens)], []
    for b, n in enumerate(lens):
        pols.append(_policies(rng, hkv, n))
        cache.set_policy(b, to_c_policies([pols[b]]))
        half = n // 2
        if half:
            cache.build(b, 0, data[b][0][:half].contiguous(), data[b][1][:half].contiguous())
        cache.append_kv(0, [b], [0, n - half], data[b][0][half:].contiguous(), data[b][1][half:].contiguous())
    assert sum(_check_codes(cache, b, 0, h, *data[b], ks, vs) for b in range(B) for h in range(hkv)) > 0
    q = W.normal((B, hq, D), 99, device="cuda")
    out, lse = cache.decode(0, list(range(B)), q)
    for b, n in enumerate(lens):
        ref = attend(q[b:b + 1].double(), _stored(data[b][0], ks), _stored(data[b][1], vs), [n - 1],
                     [pol_tuple(p) for p in pols[b]])
        check(out[b:b + 1], lse[b:b + 1], ref, 2.0 ** -11, 2.0 ** -11 if scaled else 0.0, "seq %d" % b)
    st, sl = torch.empty_like(out), torch.empty_like(lse)
    from head_aware_paged_gb300 import sp_attention_decode_static_scratch
    sp_attention_decode_static_scratch(cache.handle, 0, list(range(B)), q, st, sl)
    assert torch.equal(st, out) and torch.equal(sl, lse)
    # more sequences than the call takes, in another order, on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, l2 = cache.decode(0, [5, 0, 3], q[[5, 0, 3]].contiguous())
    side.synchronize()
    ref = [attend(q[b:b + 1].double(), _stored(data[b][0], ks), _stored(data[b][1], vs), [lens[b] - 1],
                  [pol_tuple(p) for p in pols[b]]) for b in (5, 0, 3)]
    for i in range(3):
        check(o2[i:i + 1], l2[i:i + 1], ref[i], 2.0 ** -11, 2.0 ** -11 if scaled else 0.0)
    assert cache.status() == 0


def test_special_values():
    """Infinities saturate, a NaN does not spread to its block, zeros and
    values under the least scale are zeros; nothing that reads them is non-finite."""
    gpu_ready()
    n = 40
    cache = _mk(4, 2, 16, 1, 64, 40)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G), W.HeadPolicy(G)]]))
    k, v = _kv(n, 2, 5)
    k[3, 0, 20], k[4, 1, 0], v[7, 0, 127] = float("inf"), float("-inf"), float("nan")
    v[8], k[9] = 0.0, 2.0 ** -30
    cache.build(0, 0, k, v)
    kk, vv = k.clone(), v.clone()
    vv[7, 0, 127] = 0.0                       # the NaN is not part of its block's maximum
    held = _held(cache, 0, 0, 0)
    _, sc = fp4.quantize(f64(vv[7, 0]))
    assert (held[7][3] == sc).all() and held[7][2][127] & 7 == 7
    assert held[3][1][1] == 226 and held[3][0][20] == 7
    assert (_held(cache, 0, 0, 1)[4][0][0] == 15) and (held[9][1] == 0).all() and (held[8][3] == 0).all()
    out, _ = cache.decode(0, [0], W.normal((1, 4, D), 1, device="cuda"))
    assert torch.isfinite(out).all()
    assert cache.status() == 0


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("P,hq,hkv,n,c", [(64, 32, 8, 700, 300), (16, 6, 2, 1500, 17), (128, 3, 3, 129, 128),
                                          (32, 8, 4, 33, 1), (64, 8, 2, 0, 200)])
def test_prefill_over_history(P, hq, hkv, n, c, scaled):
    gpu_ready()
    rng = np.random.default_rng(n + c)
    ns, cs = [n, n // 2, n], [c, 0, max(1, c // 3)]           # the second sequence has no rows
    cache = _mk(hq, hkv, P, 3, n + c + 700, 3 * hkv * ((n + c) // P + 4) + 8)
    ks = vs = None
    if scaled:
        ks = np.exp2(rng.uniform(-2, 2, (hkv, D))).astype(np.float32)
        vs = np.exp2(rng.uniform(-2, 2, (hkv, D))).astype(np.float32)
        cache.set_kv_scales(0, ks, vs)
    pols = [_policies(rng, hkv, n + c) for _ in range(3)]
    hist = [_kv(x, hkv, 30 + b) for b, x in enumerate(ns)]
    for b in range(3):
        cache.set_policy(b, to_c_policies([pols[b]]))
        if ns[b]:
            cache.build(b, 0, *hist[b])
    cu = [0, cs[0], cs[0], cs[0] + cs[2]]
    q = W.normal((cu[-1], hq, D), 3, device="cuda")
    k, v = _kv(cu[-1], hkv, 40)
    out, lse = cache.prefill(0, [0, 1, 2], cu, q, k, v)
    for b in (0, 2):
        sl = slice(cu[b], cu[b + 1])
        kk = torch.cat([_stored(hist[b][0], ks), k[sl].double()])
        vv = torch.cat([_stored(hist[b][1], vs), v[sl].double()])
        ref = attend(q[sl].double(), kk, vv, range(ns[b], ns[b] + cs[b]), [pol_tuple(p) for p in pols[b]])
        # with channel scales V rows are rounded to bf16 too
        check(out[sl], lse[sl], ref, 2.0 ** -8 * (2 if scaled else 1), 2.0 ** -8 if scaled else 0.0, "seq %d" % b)
    assert cache.status() == 0


@pytest.mark.parametrize("hq,hkv,P,n,pages", [(4, 2, 16, 20, 4), (2, 1, 16, 1, 1), (3, 1, 128, 200, 2), (2, 2, 32, 32, 2)])
def test_prefill_over_a_pool_smaller_than_a_tile(hq, hkv, P, n, pages):
    """Every page of a small pool in use: the last unit's tile ends behind the
    converted rows."""
    gpu_ready()
    c = 5
    cache = _mk(hq, hkv, P, 1, n + c, pages)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)] * hkv]))
    hist = _kv(n, hkv, 3)
    cache.build(0, 0, *hist)
    q = W.normal((c, hq, D), 7, device="cuda")
    k, v = _kv(c, hkv, 8)
    for cap in (None, 20.0):
        out, lse = cache.prefill(0, [0], [0, c], q, k, v, score_cap=cap)
        ref = attend(q.double(), torch.cat([_stored(hist[0]), k.double()]), torch.cat([_stored(hist[1]), v.double()]),
                     range(n, n + c), [(G, 0, 0, None)] * hkv, cap)
        check(out, lse, ref, 2.0 ** -8, 0.0, "cap %s" % cap, cap)
    assert cache.status() == 0


def test_prefill_history_converted_in_several_passes():
    """More history than the workspace's bf16 copies hold: groups of units."""
    gpu_ready()
    hq, hkv, P, n, B = 4, 4, 64, 131072, 9                    # 36 units of 64 MB in bf16, 2 GiB at a time
    cache = _mk(hq, hkv, P, B, n + 64, B * hkv * (n // P + 2))
    k, v = _kv(n, hkv, 3)
    for b in range(B):
        cache.set_policy(b, to_c_policies([[W.HeadPolicy(G)] * hkv]))
        cache.build(b, 0, torch.roll(k, b, 0).contiguous(), v)
    c = 3
    q = W.normal((B * c, hq, D), 7, device="cuda")
    kn, vn = _kv(B * c, hkv, 8)
    out, lse = cache.prefill(0, list(range(B)), [c * b for b in range(B + 1)], q, kn, vn)
    ks, vs = _stored(k), _stored(v)
    for b in (0, 4, B - 1):
        sl = slice(b * c, b * c + c)
        kk, vv = torch.cat([torch.roll(ks, b, 0), kn[sl].double()]), torch.cat([vs, vn[sl].double()])
        check(out[sl], lse[sl], attend(q[sl].double(), kk, vv, range(n, n + c), [(G, 0, 0, None)] * hkv),
              2.0 ** -8, 0.0, "seq %d" % b)
    assert cache.status() == 0


def test_serving_run():
    """A prompt in two chunks, then decode steps: unrotated projections, 4-bit
    pages, capped scores; every output against 64 bits over what the pages hold."""
    gpu_ready()
    hq, hkv, P, theta, cap = 16, 4, 32, 500000.0, 20.0
    lens, steps = [90, 333], 5
    B, tot = 2, max(lens) + steps
    cache = _mk(hq, hkv, P, B, tot + 1, B * hkv * (tot // P + 4))
    pols = [W.HeadPolicy(G), W.HeadPolicy(L, 4, 60), W.HeadPolicy(R, idx=np.arange(0, tot, 3, dtype=np.int32)),
            W.HeadPolicy(L, 0, 1)]
    pt = [pol_tuple(p) for p in pols]
    qkv = [W.normal((n + steps, hq + 2 * hkv, D), 50 + b, device="cuda") for b, n in enumerate(lens)]
    turned = [torch.tensor(np.concatenate([rope.realign(f64(x[i:i + 1, :hq + hkv]), i, theta)
                                           for i in range(x.shape[0])]), device="cuda") for x in qkv]
    for b in range(B):
        cache.set_policy(b, to_c_policies([pols]))

    def keys(b, n):
        """What the pages hold of sequence b's first n tokens, read back."""
        kk = torch.zeros(n, hkv, D, dtype=torch.float64)
        vv = torch.zeros_like(kk)
        for h in range(hkv):
            for p, (kc, kse, vc, vse) in _held(cache, b, 0, h).items():
                kk[p, h], vv[p, h] = torch.tensor(fp4.dequantize(kc, kse)), torch.tensor(fp4.dequantize(vc, vse))
        return kk.cuda(), vv.cuda()

    at = [0, 0]
    for part in range(2):
        cnt = [(n // 2 if part == 0 else n - n // 2) for n in lens]
        cu = [0, cnt[0], sum(cnt)]
        rows = torch.cat([qkv[b][at[b]:at[b] + cnt[b]] for b in range(B)])
        held = [keys(b, at[b]) for b in range(B)]
        # the chunk attends before its rows are stored: rotate into plain tensors first
        want = torch.cat([turned[b][at[b]:at[b] + cnt[b]] for b in range(B)])
        kr = want[:, hq:].to(torch.bfloat16)
        qr = want[:, :hq].to(torch.bfloat16)
        v = rows[:, hq + hkv:].contiguous()
        out, lse = cache.prefill(0, [0, 1], cu, qr, kr, v, score_cap=cap)
        got = cache.append_kv_rope(0, [0, 1], cu, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:],
                                   rope_theta=theta)
        assert ((got.double() - want[:, :hq]).abs() <= 2.0 ** -8 * want[:, :hq].abs() + 2.0 ** -18 * 4).all()
        for b in range(B):
            sl = slice(cu[b], cu[b + 1])
            kk, vv = torch.cat([held[b][0], kr[sl].double()]), torch.cat([held[b][1], v[sl].double()])
            ref = attend(qr[sl].double(), kk, vv, range(at[b], at[b] + cnt[b]), pt, cap)
            check(out[sl], lse[sl], ref, 2.0 ** -8, 0.0, "part %d seq %d" % (part, b), cap)
        at = [a + c for a, c in zip(at, cnt)]
    for s in range(steps):
        x = torch.stack([qkv[b][at[b]] for b in range(B)])
        q = cache.append_kv_rope(0, [0, 1], [0, 1, 2], x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], rope_theta=theta)
        out, lse = cache.decode(0, [0, 1], q, score_cap=cap)
        for b in range(B):
            at[b] += 1
            kk, vv = keys(b, at[b])
            check(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1].double(), kk, vv, [at[b] - 1], pt, cap),
                  2.0 ** -11, 0.0, "step %d seq %d" % (s, b), cap)
            # the stored key is the nearest code of the rotated key: within half a step of its block
            t, (kc, ksc) = at[b] - 1, _held(cache, b, 0, 0)[at[b] - 1][:2]
            ref = turned[b][t, hq].cpu().numpy()
            scl = np.repeat(fp4.SCALES[ksc], 16)
            y = np.abs(ref) / scl
            half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0)) * scl
            assert (np.abs(fp4.dequantize(kc, ksc) - ref) <= half * 1.001 + 0.07 * np.abs(ref) * (y > 5.9)).all()
    assert cache.status() == 0


def test_pack_unpack_and_realign():
    gpu_ready()
    hkv, P, n = 3, 32, 300
    src, dst = _mk(6, hkv, P, 2, 400, 100, layers=2), _mk(6, hkv, P, 2, 400, 100, layers=2)
    pols = [[W.HeadPolicy(G), W.HeadPolicy(L, 5, 70), W.HeadPolicy(R, idx=np.arange(2, n, 5, dtype=np.int32))]] * 2
    ks = np.exp2(np.random.default_rng(1).uniform(-1, 1, (hkv, D))).astype(np.float32)
    for c in (src, dst):
        for l in range(2):
            c.set_kv_scales(l, ks, ks)
    src.set_policy(1, to_c_policies(pols))
    for l in range(2):
        src.build(1, l, *_kv(n, hkv, 60 + l))
    buf = src.pack(1)
    rows = sum(len(_held(src, 1, l, h)) for l in range(2) for h in range(hkv))
    # the payload, behind the header, is 72 bytes a row and side: codes in dimension order, then scales
    payload = buf.cpu().numpy()[-2 * 72 * rows:]
    first = _held(src, 1, 0, 0)
    for p in (0, 17, n - 1):
        code, sc = first[p][:2]
        assert (payload[72 * p:72 * p + 64] == (code[0::2] | (code[1::2] << 4))).all()
        assert (payload[72 * p + 64:72 * p + 72] == sc).all()
    dst.unpack(0, buf)
    for l in range(2):
        for h in range(hkv):
            a, b = _held(src, 1, l, h), _held(dst, 0, l, h)
            assert sorted(a) == sorted(b)
            for p in a:
                assert all((x == y).all() for x, y in zip(a[p], b[p]))
    # realign layer 1, head 0, positions [10, 200): dequantise, rotate, quantise again
    before = _held(dst, 0, 1, 0)
    others = _held(dst, 0, 1, 1)
    dst.rope_realign(1, [0], 1234567, kv_head=0, pos_lo=10, pos_hi=200)
    after = _held(dst, 0, 1, 0)
    for p in before:
        if not 10 <= p < 200:
            assert all((x == y).all() for x, y in zip(before[p], after[p]))
            continue
        x = rope.realign(fp4.dequantize(*before[p][:2], ks[0])[None], 1234567)[0] / ks[0]
        s = np.repeat(fp4.SCALES[after[p][1]], 16)
        b = np.abs(x).reshape(8, 16).max(1) / 6
        assert (np.abs(fp4.SCALES[after[p][1]] / b - 1) <= 2.0 ** -4 + 1e-5).all()
        y = np.abs(x) / s
        half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0)) * s
        assert (np.abs(fp4.dequantize(*after[p][:2]) - x) <= half * 1.001 + 0.07 * np.abs(x) * (y > 5.9)).all()
        assert all((u == w).all() for u, w in zip(before[p][2:], after[p][2:]))
    assert all(all((x == y).all() for x, y in zip(others[p], t)) for p, t in _held(dst, 0, 1, 1).items())
    assert src.status() == 0 and dst.status() == 0


def test_bytes_and_refusals():
    gpu_ready()
    from head_aware_paged_gb300 import KV_FP4, Config, SegPagedError, sp_required_bytes
    base = dict(num_layers=1, num_q_heads=4, num_kv_heads=2, head_dim=128, page_size=64, max_seqs=1,
                max_seq_len=256, num_pages=16, kv_dtype=KV_FP4)
    assert sp_required_bytes(Config(**base))[0] == 2 * 16 * 64 * 72
    with pytest.raises(SegPagedError) as e:
        sp_required_bytes(Config(**dict(base, head_dim=64)))
    assert e.value.status == 3
    cache = _mk(4, 2, 16, 1, 256, 64)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G), W.HeadPolicy(L, 4, 8)]]))
    with pytest.raises(SegPagedError):
        cache.decode(0, [0], W.normal((1, 4, D), 1, device="cuda"))     # nothing appended
    cache.build(0, 0, *_kv(100, 2, 1))
    assert cache.count_decode_bytes(0, [0], [99]) == (100 + 12) * 2 * 72
    with pytest.raises(SegPagedError):                                  # scales are fixed once pages hold codes
        cache.set_kv_scales(0, np.ones((2, D)), np.ones((2, D)))
    assert cache.status() == 0


def test_graph_replay():
    """A captured prefill and decode, replayed, give what the calls gave."""
    gpu_ready()
    hq, hkv, n = 8, 2, 500
    cache = _mk(hq, hkv, 64, 2, 600, 60)
    for b in range(2):
        cache.set_policy(b, to_c_policies([[W.HeadPolicy(G), W.HeadPolicy(L, 4, 100)]]))
        cache.build(b, 0, *_kv(n, hkv, b))
    q, k, v = W.normal((40, hq, D), 1, device="cuda"), *_kv(40, hkv, 9)
    qd = q[:2].clone()
    want = [*cache.prefill(0, [0, 1], [0, 30, 40], q, k, v), *cache.decode(0, [0, 1], qd)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = [*cache.prefill(0, [0, 1], [0, 30, 40], q, k, v), *cache.decode(0, [0, 1], qd)]
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cache.status() == 0


@pytest.mark.parametrize("cap", [None, 50.0])
@pytest.mark.parametrize("hq,hkv,P", [(8, 2, 64), (24, 2, 16), (3, 3, 32)])
@pytest.mark.parametrize("which,qs", [("least", 0.05), ("least", 600.0), ("largest", 0.05), ("largest", 600.0),
                                      ("mixed", 1.0), ("none", 1e-6), ("none", 1e6)])
def test_decode_at_the_ends_of_the_scale_range(which, qs, hq, hkv, P, cap):
    """Channel scales of 2^-14 and 128 and everything between, small and large
    queries.  Powers of two, so that query times scale has bf16's 8 bits: it
    enters the products exactly, but for elements 2^-28 below the head's largest
    (mixed scales: 2^-11 of each product is allowed)."""
    gpu_ready()
    rng = np.random.default_rng(3)
    ex = {"least": np.full((hkv, D), -14), "largest": np.full((hkv, D), 7), "mixed": rng.integers(-14, 8, (hkv, D)),
          "none": np.zeros((hkv, D), int)}[which]
    ks = np.exp2(ex).astype(np.float32)
    lens = [1, 2, 3, 70, 500]
    cache = _mk(hq, hkv, P, len(lens), 512, len(lens) * hkv * (512 // P + 2))
    if which != "none":
        cache.set_kv_scales(0, ks, np.ones((hkv, D), np.float32))
    data = [_kv(n, hkv, 80 + b) for b, n in enumerate(lens)]
    for b in range(len(lens)):
        cache.set_policy(b, to_c_policies([[W.HeadPolicy(G)] * hkv]))
        cache.build(b, 0, *data[b])
    q = (W.normal((len(lens), hq, D), 99, device="cuda").float() * qs).to(torch.bfloat16)
    out, lse = cache.decode(0, list(range(len(lens))), q, score_cap=cap)
    for b, n in enumerate(lens):
        ref = attend(q[b:b + 1].double(), _stored(data[b][0], ks), _stored(data[b][1]), [n - 1], [(G, 0, 0, None)] * hkv, cap)
        check(out[b:b + 1], lse[b:b + 1], ref, 2.0 ** -11, 2.0 ** -11 if which == "mixed" else 0.0, "seq %d" % b, cap)
    assert cache.status() == 0


@pytest.mark.parametrize("rope_path", [False, True])
def test_scale_beside_a_tie(rope_path):
    """Block maxima that are the fp32 number just below 6 * 19/16 (times a power
    of two): amax / 6 lies below the tie of two scales, its nearest is 9/8.  They
    come about as x * fp32(1 / channel scale), x and the scale searched for here."""
    gpu_ready()
    below = np.nextafter(np.float32(7.125), np.float32(0))
    pairs = []
    for m in range(128, 256):
        x = np.float32(m / 128)
        want = np.float32(float(below) / float(x))
        for c in (want, np.nextafter(want, np.float32(0)), np.nextafter(want, np.float32(99))):
            s = np.float32(1.0 / float(c))
            for t in (s, np.nextafter(s, np.float32(0)), np.nextafter(s, np.float32(9))):
                if x * (np.float32(1) / t) == below and len(pairs) < 8 and (not pairs or pairs[-1][0] != x):
                    pairs.append((x, t))
    assert len(pairs) == 8
    cache = _mk(2, 1, 16, 1, 64, 8)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    s = np.ones((1, D), np.float32)
    n = 24                                       # powers of two from 2^-12 (subnormal scales) to 2^11
    k = np.zeros((n, 1, D), np.float32)
    for b, (x, t) in enumerate(pairs):
        s[0, 16 * b + 3] = t
        k[:, 0, 16 * b + 3] = x * np.exp2(np.arange(n) - 12)
    cache.set_kv_scales(0, s, s)
    kt = torch.tensor(k, device="cuda").to(torch.bfloat16)
    if rope_path:                                # no rotation: frequency 0
        cache.append_kv_rope(0, [0], [0, n], None, kt, kt, inv_freq=[0.0] * (D // 2))
    else:
        cache.append_kv(0, [0], [0, n], kt, kt)
    sc = fp4.quantize(f64(kt[:, 0]), s[0])[1]
    assert (sc[12] == (15 << 3) + 1).all()       # 9/8
    assert _check_codes(cache, 0, 0, 0, kt, kt, s, s) == n
    assert cache.status() == 0


@pytest.mark.parametrize("at", [0, 40, 63])
def test_weights_far_below_the_largest(at):
    """One key e^18 times as heavy as the 63 others of its item, its value zero:
    the output is theirs alone.  P keeps weights down to half of 2^-24 of 2^7,
    2^-32 of the largest (a reference at the maximum itself would drop them)."""
    gpu_ready()
    n = 64
    cache = _mk(2, 1, 64, 1, 128, 4)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = torch.zeros(n, 1, D, dtype=torch.bfloat16, device="cuda")
    k[at, 0, 0] = 6.0
    v = torch.full_like(k, 6.0)
    v[at] = 0.0
    cache.build(0, 0, k, v)
    q = torch.zeros(1, 2, D, dtype=torch.bfloat16, device="cuda")
    q[0, :, 0] = 34.0                            # 34 * 6 / sqrt(128) = 18.03
    out, lse = cache.decode(0, [0], q)
    o, z, A, _, S = attend(q.double(), _stored(k), _stored(v), [n - 1], [(G, 0, 0, None)])
    tol = 2.0 ** -8 * o + 2.0 ** -14 * A + 2.0 ** -32 * S
    assert (o > 4e-6).all() and ((out.double() - o).abs() <= tol).all()
    assert ((lse.double() - z).abs() <= 2.0 ** -19 * (1 + z)).all()
    assert cache.status() == 0


def test_offsets_past_32_bits():
    """A pool whose K half is longer than 4 GiB, read and written at its end."""
    gpu_ready()
    hq, hkv, P, n, B = 8, 2, 64, 131072, 234
    pages = B * hkv * (n // P) + 8
    assert (pages - 8) * P * 72 > 1 << 32
    cache = _mk(hq, hkv, P, B, n + 64, pages, batch=2)
    k, v = _kv(n, hkv, 3)
    for b in range(B):
        cache.set_policy(b, to_c_policies([[W.HeadPolicy(G)] * hkv]))
        cache.build(b, 0, k if b < B - 1 else torch.roll(k, 1, 0).contiguous(), v)
    ids = cache.export_table(B - 1, 0, hkv - 1)[0]
    assert min(ids) * P * 72 >= 1 << 32
    ks, vs = torch.roll(_stored(k), 1, 0), _stored(v)
    pol = [(G, 0, 0, None)] * hkv
    q = W.normal((3, hq, D), 7, device="cuda")
    out, lse = cache.decode(0, [B - 1], q[:1].contiguous())
    check(out, lse, attend(q[:1].double(), ks, vs, [n - 1], pol), 2.0 ** -11, 0.0, "decode")
    kn, vn = _kv(3, hkv, 8)
    out, lse = cache.prefill(0, [B - 1], [0, 3], q, kn, vn)
    check(out, lse, attend(q.double(), torch.cat([ks, kn.double()]), torch.cat([vs, vn.double()]), range(n, n + 3), pol),
          2.0 ** -8, 0.0, "prefill")
    low = cache.k_pool()[:64].clone()
    cache.append_kv_rope(0, [B - 1], [0, 3], None, kn, vn, inv_freq=[0.0] * 64)         # a new page, no rotation
    ks, vs = torch.cat([ks, _stored(kn)]), torch.cat([vs, _stored(vn)])
    out, lse = cache.decode(0, [B - 1], q[2:].contiguous())
    check(out, lse, attend(q[2:].double(), ks, vs, [n + 2], pol), 2.0 ** -11, 0.0, "after the write")
    assert torch.equal(cache.k_pool()[:64], low)
    assert cache.status() == 0


def test_two_graphs_share_the_workspace():
    """Two captured steps of one cache, replayed in turns in stream order, give
    what the calls gave: no state is left in the workspace."""
    gpu_ready()
    hq, hkv = 8, 2
    cache = _mk(hq, hkv, 16, 3, 3000, 3 * hkv * 200)
    for b, n in enumerate((2500, 31, 700)):
        cache.set_policy(b, to_c_policies([[W.HeadPolicy(G), W.HeadPolicy(L, 4, 300)]]))
        cache.build(b, 0, *_kv(n, hkv, b))
    q, k, v = W.normal((40, hq, D), 1, device="cuda"), *_kv(40, hkv, 9)
    calls = [lambda: [*cache.decode(0, [0, 1, 2], q[:3].contiguous(), score_cap=30.0), *cache.prefill(0, [1], [0, 40], q, k, v)],
             lambda: [*cache.prefill(0, [2, 0], [0, 17, 40], q, k, v), *cache.decode(0, [2], q[7:8].contiguous())]]
    want = [[x.clone() for x in c()] for c in calls]
    s = torch.cuda.Stream()
    graphs, got = [], []
    for c in calls:
        s.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            got.append(c())
    for i in (0, 1, 1, 0, 0, 1):
        for t in got[i]:
            t.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    assert cache.status() == 0
