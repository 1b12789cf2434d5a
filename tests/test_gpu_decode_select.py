"""GPU: page bounds and the decode over chosen pages.

Bounds and kept pages are integer results: they equal the oracle's
(oracle/choose.py) on the keys as the pages hold them, bit for bit.  Outputs are
compared with attention in 64 bits over the kept pages' tokens, within the
tolerances of the decode over those pages (_attn64.check)."""
import numpy as np
import pytest
import torch

import workloads as W
from _attn64 import attend, check
from _gpu_common import gpu_ready, to_c_policies
from oracle import choose, fp4

pytestmark = pytest.mark.gpu

G, L, R = W.GLOBAL, W.LOCAL, W.RETRIEVAL


def _mk(hq, hkv, d, P, seqs, max_len, pages=None, kv="bf16", layers=1, batch=None, attach=True):
    import head_aware_paged_gb300 as H
    c = H.SegPagedCache(H.Config(num_layers=layers, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P,
                                 max_seqs=seqs, max_seq_len=max_len,
                                 num_pages=pages or seqs * layers * hkv * (max_len // P + 2), max_idx_per_seq=8192,
                                 max_tokens=max_len, max_batch=batch or seqs,
                                 kv_dtype={"bf16": H.KV_BF16, "fp8": H.KV_FP8, "fp4": H.KV_FP4}[kv]))
    if attach:
        c.attach_page_bounds()
    return c


def _fp4_rows(groups, value):
    """The values code * block scale of groups [n, 1152] (uint8), as [n * 16, 128]."""
    out = np.zeros((len(groups), 16, 128), np.float32)
    place = np.arange(1152)
    for slot in range(16):
        for b in range(8):                                    # (the places that the oracle's reader takes)
            if value:
                at, sc = slot * 64 + (b ^ (4 if slot % 4 >= 2 else 0)) * 8, 1024 + 16 * b + 4 * (slot % 4) + slot // 4
            else:
                r = fp4.k_row(slot)
                at, sc = r * 64 + b * 8, 1024 + 16 * (r % 8) + 4 * (b // 2) + 2 * (r // 8) + b % 2
            byte = groups[:, place[at:at + 8]]
            code = np.stack([byte & 15, byte >> 4], -1).reshape(len(groups), 16)
            v = np.where(code & 8, -1.0, 1.0) * fp4.E2M1[code & 7]
            out[:, slot, 16 * b:16 * b + 16] = v * fp4.SCALES[groups[:, sc]][:, None]
    return out.reshape(-1, 128)


def _stored(c, seq, h, which=0, layer=0, scale=None):
    """Positions and rows [n, d] (float32 values, as float64) that a unit's pages hold, by position."""
    import head_aware_paged_gb300 as H
    ids, pos = c.export_table(seq, layer, h)
    if not ids:
        return np.zeros(0, np.int64), np.zeros((0, c.cfg.head_dim))
    pool = (c.k_pool() if which == 0 else c.v_pool())[torch.tensor(ids, device="cuda")].cpu()
    if c.cfg.kv_dtype == H.KV_FP4:
        x = _fp4_rows(pool.reshape(-1, 1152).numpy(), which == 1)
    elif c.cfg.kv_dtype == H.KV_FP8:
        x = pool.view(torch.float8_e4m3fn).float().numpy()
    else:
        x = pool.float().numpy()
    x = x.astype(np.float32)
    if scale is not None:
        x = x * np.asarray(scale, np.float32)
    at = np.array(pos).reshape(-1)
    order = np.argsort(at[at >= 0], kind="stable")
    return at[at >= 0][order], x.reshape(-1, c.cfg.head_dim)[at >= 0][order].astype(np.float64)


def _check_bounds(c, seqs, heads, scale=None, layer=0):
    """Bounds of every full page of the GLOBAL heads; returns {(seq, head): per page bounds}."""
    codes, step = (x.cpu().numpy() for x in c.page_bounds())
    P, res = c.cfg.page_size, {}
    for s in seqs:
        for h in heads:
            ids, _ = c.export_table(s, layer, h)
            at, k = _stored(c, s, h, 0, layer, None if scale is None else scale[h])
            assert (at == np.arange(len(at))).all()
            res[s, h] = []
            for j in range(len(at) // P):
                hi, lo, st = choose.bounds(k[j * P:(j + 1) * P])
                assert step[ids[j]] == st, (s, h, j)
                assert (codes[ids[j], 0] == hi).all() and (codes[ids[j], 1] == lo).all(), (s, h, j)
                res[s, h].append((hi, lo, st))
    return res


def _want_pages(q, pages, n, P, first, newest, top):
    nb = -(-n // P)
    if nb <= first + newest + top:
        return list(range(nb))
    sc = choose.scores(q, pages)
    return choose.kept(sc + [0.0] * (nb - len(sc)), nb, first, newest, top)


def _check_select(c, seqs, pols, q, top, first, newest, cap=None, scales=None, layer=0, what="", res=None):
    """decode_select against the oracle; returns its outputs."""
    hkv, P, d = c.cfg.num_kv_heads, c.cfg.page_size, c.cfg.head_dim
    g = c.cfg.num_q_heads // hkv
    out, lse, pages = res or c.decode_select(layer, seqs, q, top, first, newest, score_cap=cap)
    assert c.status() == 0
    glob = [h for h in range(hkv) if pols[h].kind == G]
    bounds = _check_bounds(c, seqs, glob, None if scales is None else scales[0], layer)
    got = pages.cpu().numpy()
    qd = q.double().cpu()
    kv = c.cfg.kv_dtype
    for b, s in enumerate(seqs):
        n = c.seq_len(s, layer)
        ks, vs, rule = torch.zeros(n, hkv, d, dtype=torch.float64), torch.zeros(n, hkv, d, dtype=torch.float64), []
        for h in range(hkv):
            for which, x in ((0, ks), (1, vs)):
                at, rows = _stored(c, s, h, which, layer, None if scales is None else scales[which][h])
                keep = at < n
                x[torch.from_numpy(at[keep]), h] = torch.from_numpy(rows[keep])
            if h in glob:
                want = _want_pages(qd[b, h * g:h * g + g].numpy(), bounds[s, h], n, P, first, newest, top)
                assert got[b, h].tolist() == want + [-1] * (first + newest + top - len(want)), (what, s, h)
                tok = (np.array(want, np.int64)[:, None] * P + np.arange(P)).ravel()
                rule.append((R, 0, 0, tok[tok < n]))
            else:
                assert (got[b, h] == -1).all()
                p = pols[h]
                rule.append((p.kind, p.sink, p.window, p.idx if p.idx is not None else ()))
        ref = attend(qd[b:b + 1], ks, vs, [n - 1], rule, cap)
        # bf16 pages: P in bf16; others: P, and the query under channel scales, in f16
        check(out[b:b + 1].cpu(), lse[b:b + 1].cpu(), ref, 2.0 ** -8 if kv == 0 else 2.0 ** -11,
              0.0 if kv == 0 else 2.0 ** -11, "%s seq %d" % (what, s), cap)
    return out, lse, pages


def _keys(n, hkv, d, seed, device="cuda"):
    """Keys that drift, so that pages differ."""
    x = W.normal((n, hkv, d), seed, device=device).float()
    y = W.normal((n // 24 + 1, hkv, d), seed + 1, device=device).float()
    return (x * 0.5 + y.repeat_interleave(24, 0)[:n]).to(torch.bfloat16)


def _classes(hkv):
    return [W.HeadPolicy(G), W.HeadPolicy(L, 4, 60), W.HeadPolicy(G), W.HeadPolicy(R, idx=np.arange(3, 3000, 7, dtype=np.int32)),
            W.HeadPolicy(R, idx=np.zeros(0, np.int32)), W.HeadPolicy(G), W.HeadPolicy(L, 0, 1), W.HeadPolicy(G)][:hkv]


SHAPES = [("bf16", 128, 64, 8, 2), ("bf16", 64, 16, 6, 3), ("bf16", 128, 128, 7, 1), ("bf16", 64, 32, 16, 1),
          ("bf16", 128, 16, 40, 8), ("fp8", 128, 32, 20, 5), ("fp8", 128, 128, 4, 4), ("fp8", 128, 16, 6, 6),
          ("fp4", 128, 64, 32, 8), ("fp4", 128, 16, 12, 3), ("fp4", 128, 128, 12, 1), ("fp4", 128, 32, 5, 5)]


@pytest.mark.parametrize("kv,d,P,hq,hkv", SHAPES)
def test_pages_and_outputs(kv, d, P, hq, hkv):
    """Lengths from one token on, chosen pages of every count, ragged."""
    gpu_ready()
    pols = _classes(hkv)
    lens = [1, P - 1, P, P + 1, 6 * P + 5, 21 * P, 40 * P - 1]
    c = _mk(hq, hkv, d, P, len(lens), 41 * P, kv=kv)
    rng = np.random.default_rng(P + hq)
    scales = None
    if kv != "bf16":
        scales = np.exp2(rng.integers(-3, 3, (2, hkv, d))).astype(np.float32)
        c.set_kv_scales(0, scales[0], scales[1])
    for s, n in enumerate(lens):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(n, hkv, d, 10 * s), W.normal((n, hkv, d), 10 * s + 5, device="cuda"))
    ids = [3, 0, 6, 1, 5, 2, 4]
    q = W.normal((len(ids), hq, d), 99, device="cuda")
    for top, first, newest in ((4, 1, 1), (0, 0, 1), (0, 2, 3), (7, 0, 2), (1, 0, 1), (30, 3, 7), (200, 1, 1)):
        _check_select(c, ids, pols, q, top, first, newest, scales=scales, what="%d %d %d" % (top, first, newest))
    _check_select(c, ids, pols, q, 5, 1, 2, cap=20.0, scales=scales, what="capped")


@pytest.mark.parametrize("kv,seqs,hq,hkv", [("bf16", 1, 16, 8), ("bf16", 2, 5, 5), ("bf16", 5, 72, 8), ("bf16", 12, 16, 8),
                                            ("bf16", 27, 8, 8), ("bf16", 40, 24, 8), ("fp8", 6, 8, 8), ("fp8", 31, 16, 8),
                                            ("fp4", 3, 24, 8), ("fp4", 20, 16, 8), ("fp4", 33, 72, 8)])
def test_batches(kv, seqs, hq, hkv):
    """From one unit to hundreds (blocks and warps a unit differ), ragged."""
    gpu_ready()
    P, rng = 16, np.random.default_rng(seqs)
    pols = _classes(hkv)
    lens = [int(x) for x in rng.integers(1, 500, seqs)]
    lens[0] = 1100
    c = _mk(hq, hkv, 128, P, seqs, 1200, pages=seqs * hkv * 34 + hkv * 40, kv=kv)
    for s, n in enumerate(lens):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(n, hkv, 128, 10 * s), W.normal((n, hkv, 128), 10 * s + 5, device="cuda"))
    ids = [int(x) for x in rng.permutation(seqs)]
    q = W.normal((seqs, hq, 128), 99, device="cuda")
    _check_select(c, ids, pols, q, 6, 1, 2, cap=30.0 if seqs % 3 == 0 else None)


@pytest.mark.parametrize("kv,P", [("bf16", 64), ("fp8", 16), ("fp4", 32)])
def test_all_pages_kept(kv, P):
    """More pages asked for than there are: plain attention over everything that
    is seen; the outputs do not depend on which of them are asked for."""
    gpu_ready()
    hkv, hq, d = 8, 32, 128
    pols = _classes(hkv)
    c = _mk(hq, hkv, d, P, 2, 1000, kv=kv)
    for s in range(2):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(700 + 200 * s, hkv, d, s), W.normal((700 + 200 * s, hkv, d), s + 5, device="cuda"))
    q = W.normal((2, hq, d), 9, device="cuda")
    for cap in (None, 30.0):
        want = _check_select(c, [0, 1], pols, q, 1000, 1, 1, cap=cap)
        got = c.decode_select(0, [0, 1], q, 1000, score_cap=cap, want_pages=False, want_lse=False)
        assert torch.equal(got[0], want[0]) and got[1] is None and got[2] is None


@pytest.mark.parametrize("d,group", [(128, 1), (64, 16), (128, 16)])
def test_ties_take_the_lower_page(d, group):
    """Every page the same keys, but a few better ones: equal scores everywhere."""
    gpu_ready()
    P, nb = 16, 600
    c = _mk(group, 1, d, P, 1, nb * P)
    c.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = W.normal((P, 1, d), 3, device="cuda").repeat(nb, 1, 1)
    q = W.normal((1, group, d), 4, device="cuda")
    best = q[0, 0].float() * 4
    for j in (17, 300, 599, 598):
        k[j * P] = best.to(torch.bfloat16)
    c.build(0, 0, k, k)
    for top in (1, 2, 3, 50, 257, 596):
        _check_select(c, [0], [W.HeadPolicy(G)], q, top, 1, 2, what="top %d" % top)


def test_long_unit_and_its_neighbours():
    """More candidates than a block has threads or a list holds in shared memory."""
    gpu_ready()
    P, n = 16, 200003
    c = _mk(2, 1, 64, P, 2, n)
    for s in range(2):
        c.set_policy(s, to_c_policies([[W.HeadPolicy(G)]]))
        m = n if s == 0 else 1000
        c.build(s, 0, _keys(m, 1, 64, s), W.normal((m, 1, 64), s + 5, device="cuda"))
    q = W.normal((2, 2, 64), 9, device="cuda")
    for top in (1, 100, 9000):
        out, lse, pages = c.decode_select(0, [0, 1], q, top, 2, 3)
        k = _stored(c, 0, 0)[1].reshape(-1)[:n // P * P * 64].reshape(-1, P, 64)
        hi, lo = k.max(1), k.min(1)
        st = choose.grid(np.maximum(abs(hi), abs(lo)))
        up, dn = np.ceil(hi / st[:, None]), np.floor(lo / st[:, None])
        sc = np.full(len(st), -np.inf)
        for r in range(2):
            x, t = choose.query(q[0, r].double().cpu().numpy())
            sc = np.maximum(sc, np.maximum(x * up, x * dn).sum(1) * st * t)
        nb = -(-n // P)
        want = choose.kept(sc.tolist() + [0.0], nb, 2, 3, top)
        assert pages[0, 0].tolist() == want
        small = _want_pages(q[1].double().cpu().numpy(), _check_bounds(c, [1], [0])[1, 0], 1000, P, 2, 3, top)
        assert pages[1, 0].tolist() == small + [-1] * (top + 5 - len(small))
        tok = torch.tensor(want)[:, None] * P + torch.arange(P)
        tok = tok[tok < n]
        ks, vs = (torch.from_numpy(_stored(c, 0, 0, w)[1])[tok][:, None] for w in (0, 1))
        ref = attend(q[:1].double().cpu(), ks, vs, [len(tok) - 1], [(G, 0, 0, None)])
        check(out[:1].cpu(), lse[:1].cpu(), ref, 2.0 ** -8, 0.0, "top %d" % top)
    assert c.status() == 0


@pytest.mark.parametrize("kv,d,hq,hkv,cap", [("bf16", 64, 3, 1, None), ("bf16", 128, 12, 1, 30.0), ("fp8", 128, 4, 2, None),
                                            ("fp8", 128, 16, 1, 30.0), ("fp4", 128, 8, 1, 30.0), ("fp4", 128, 24, 2, None)])
def test_many_pages_kept(kv, d, hq, hkv, cap):
    """More pages kept than a cluster's list holds: the choice in a launch of its own,
    next to a sequence that keeps everything and LOCAL heads."""
    gpu_ready()
    P, lens = 16, [35000, 900, 1]
    pols = [W.HeadPolicy(G), W.HeadPolicy(L, 4, 60)][:hkv]
    c = _mk(hq, hkv, d, P, 3, 36000, pages=hkv * 2400, kv=kv)
    scales = None
    if kv != "bf16":
        scales = np.exp2(np.random.default_rng(3).integers(-3, 3, (2, hkv, d))).astype(np.float32)
        c.set_kv_scales(0, scales[0], scales[1])
    for s, n in enumerate(lens):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(n, hkv, d, 10 * s), W.normal((n, hkv, d), 10 * s + 5, device="cuda"))
    q = W.normal((3, hq, d), 99, device="cuda")
    _check_select(c, [1, 0, 2], pols, q, 2060, 1, 2, cap=cap, scales=scales)
    again = c.decode_select(0, [1, 0, 2], q, 2060, 1, 2, score_cap=cap)
    few = c.decode_select(0, [0], q[1:2].contiguous(), 2060, 1, 2, score_cap=cap)
    assert torch.equal(again[2][1], few[2][0])


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_one_heavy_head_among_light_ones(kv):
    """One GLOBAL head of each of 24 sequences keeps many pages, the others read a
    few rows: shared out page by page instead of unit by unit."""
    gpu_ready()
    P, hkv, hq = 32, 8, 16
    pols = [W.HeadPolicy(G) if h == 3 else W.HeadPolicy(L, 4, 60) for h in range(hkv)]
    lens = [6000 + 10 * s for s in range(24)]
    c = _mk(hq, hkv, 128, P, 24, 6400, pages=24 * 300, kv=kv)
    for s, n in enumerate(lens):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(n, hkv, 128, 10 * s), W.normal((n, hkv, 128), 10 * s + 5, device="cuda"))
    q = W.normal((24, hq, 128), 99, device="cuda")
    out, lse, pages = c.decode_select(0, list(range(24)), q, 160, 1, 2)
    for s in (0, 11, 23):
        _check_select(c, [s], pols, q[s:s + 1], 160, 1, 2, what=str(s), res=(out[s:s + 1], lse[s:s + 1], pages[s:s + 1]))


@pytest.mark.parametrize("kv,d,P,hq,hkv", [("bf16", 64, 16, 4, 2), ("bf16", 128, 64, 9, 3), ("fp8", 128, 32, 9, 3),
                                           ("fp4", 128, 16, 9, 3)])
def test_bounds_follow_every_write(kv, d, P, hq, hkv):
    """build, append, token by token over a page's end, the rope forms over held
    tokens, realignment of a range, release and other sequences in the same
    pages, pack and unpack: after each the bounds of all full pages are those of
    the keys that the pages hold."""
    gpu_ready()
    pols = [W.HeadPolicy(G), W.HeadPolicy(L, 4, 60), W.HeadPolicy(G)][:hkv]
    glob = [h for h in range(hkv) if pols[h].kind == G]
    c = _mk(hq, hkv, d, P, 4, 20 * P, pages=3 * hkv * 21, kv=kv, layers=1)
    scale = None
    if kv != "bf16":
        scale = np.random.default_rng(1).uniform(0.25, 4.0, (hkv, d)).astype(np.float32)
        c.set_kv_scales(0, scale, scale)
    for s in range(4):
        c.set_policy(s, to_c_policies([pols]))
    x = lambda n, seed: (_keys(n, hkv, d, seed), W.normal((n, hkv, d), seed + 7, device="cuda"))  # noqa: E731
    c.build(0, 0, *x(5 * P + 3, 1))
    _check_bounds(c, [0], glob, scale)
    c.append_kv(0, [0, 1], [0, 2 * P, 2 * P + 1], *x(2 * P + 1, 2))
    _check_bounds(c, [0, 1], glob, scale)
    for i in range(P + 2):
        k, v = x(2, 50 + i)
        c.append_kv(0, [1, 0], [0, 1, 2], k, v)
    _check_bounds(c, [0, 1], glob, scale)
    k, v = x(P + 5, 3)
    c.append_kv_rope(0, [0], [0, P + 5], None, k, v, pos=[2 * P - 2])
    _check_bounds(c, [0], glob, scale)
    p = torch.randint(0, 1000, (3, 3 * P), device="cuda")
    k, v = x(3 * P, 4)
    c.append_kv_rope_axes(0, [0, 1], [0, 2, 3 * P], None, k, v, p, [i % 3 for i in range(d // 2)], pos=[P - 1, P])
    _check_bounds(c, [0, 1], glob, scale)
    c.rope_realign(0, [0, 1], 77, pos_lo=P // 2, pos_hi=3 * P + 1)
    _check_bounds(c, [0, 1], glob, scale)
    c.rope_realign(0, [0], -5, kv_head=glob[-1])
    _check_bounds(c, [0, 1], glob, scale)
    buf = c.pack(0)
    c.release(0)
    c.append_kv(0, [2], [0, 7 * P + 1], *x(7 * P + 1, 5))       # takes the released pages
    c.unpack(3, buf)
    _check_bounds(c, [1, 2, 3], glob, scale)
    assert c.status() == 0


def test_other_layers_and_sequences_keep_their_bounds():
    gpu_ready()
    c = _mk(4, 2, 128, 32, 2, 400, layers=3)
    pol = [[W.HeadPolicy(G), W.HeadPolicy(G)]] * 3
    for s in range(2):
        c.set_policy(s, to_c_policies(pol))
        for layer in range(3):
            c.build(s, layer, _keys(300 + layer, 2, 128, 10 * s + layer), W.normal((300 + layer, 2, 128), 4, device="cuda"))
    q = W.normal((2, 4, 128), 5, device="cuda")
    for layer in (1, 0, 2):
        _check_select(c, [1, 0], pol[0], q, 3, 1, 1, layer=layer, what="layer %d" % layer)


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_unusual_keys_and_queries(kv):
    """Zeros, one huge channel, tiny and huge magnitudes, one token that stands out; queries of
    zeros, of one element, tiny and huge."""
    gpu_ready()
    P, d = 16, 128
    c = _mk(4, 1, d, P, 1, 400, kv=kv)
    c.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = _keys(390, 1, d, 1)
    k[0:32] = 0
    k[32:48, :, 5] = 300.0
    k[48:64] *= 2.0 ** -12
    k[64:80] *= 2.0 ** 5
    k[100] = -9.0
    k[112:128] = 127.0 / 64
    k[128:144] = 128.0 / 64
    k[144:160] = -k[144:160].abs()
    c.build(0, 0, k, W.normal((390, 1, d), 3, device="cuda"))
    q = W.normal((1, 4, d), 9, device="cuda")
    q[0, 1] = 0
    q[0, 2, 1:] = 0
    q[0, 3] *= 2.0 ** -20
    for top in (1, 6, 12):
        _check_select(c, [0], [W.HeadPolicy(G)], q, top, 1, 1, what=str(top))
    _check_select(c, [0], [W.HeadPolicy(G)], torch.zeros_like(q), 5, 0, 1, what="zero")


def test_infinite_steps_and_nan():
    """Bounds and choice stay defined at the grid's ends: magnitudes past 127 * 2^50
    saturate, NaN keys do not count, and a NaN in a query stays in its rows."""
    gpu_ready()
    P, d = 16, 64
    c = _mk(2, 2, d, P, 1, 200)
    pol = [W.HeadPolicy(G), W.HeadPolicy(G)]
    c.set_policy(0, to_c_policies([pol]))
    k = _keys(180, 2, d, 1)
    k[16:32, 0, 3] = 3e38
    k[32:48, 0, 4] = -3e38
    k[48:64, 0] *= 1e-30
    c.build(0, 0, k, W.normal((180, 2, d), 3, device="cuda"))
    q = W.normal((1, 2, d), 9, device="cuda")
    bounds = _check_bounds(c, [0], [0, 1])
    _, _, pages = c.decode_select(0, [0], q, 4)
    for h in range(2):
        assert pages[0, h].tolist() == _want_pages(q[0, h:h + 1].double().cpu().numpy(), bounds[0, h], 180, P, 1, 1, 4)
    clean = c.decode_select(0, [0], q, 4)
    bad = q.clone()
    bad[0, 0, 7] = float("nan")
    out, lse, pages = c.decode_select(0, [0], bad, 4)
    assert torch.isnan(out[0, 0]).all() and torch.equal(out[0, 1], clean[0][0, 1])
    assert torch.equal(pages[0, 1], clean[2][0, 1]) and c.status() == 0
    got = pages[0, 0].tolist()
    assert got == sorted(set(got)) and 0 <= got[0] and got[-1] == 11


def test_nan_keys_do_not_count():
    """In one dimension of some rows, and of every row."""
    gpu_ready()
    P, d = 32, 128
    c = _mk(1, 1, d, P, 1, 100)
    c.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = _keys(96, 1, d, 1)
    k[3:9, 0, 5] = float("nan")
    k[32:64, 0, 6] = float("nan")
    c.build(0, 0, k, k)
    codes, step = (x.cpu().numpy() for x in c.page_bounds())
    ids, _ = c.export_table(0, 0, 0)
    x = k[:, 0].double().cpu().numpy()
    for j, fix in ((0, x[0, 5]), (1, 0.0)):
        rows = np.where(np.isnan(x[j * P:(j + 1) * P]), fix, x[j * P:(j + 1) * P])
        hi, lo, s = choose.bounds(rows)
        assert step[ids[j]] == s and (codes[ids[j], 0] == hi).all() and (codes[ids[j], 1] == lo).all()


def test_captured_decode_and_write():
    """A step in a graph: held tokens written again, then the decode; replayed with
    other inputs, and after the sequences grew past the page of the written token."""
    gpu_ready()
    hq, hkv, d, P = 8, 2, 128, 16
    pols = [W.HeadPolicy(G), W.HeadPolicy(L, 4, 60)]
    c = _mk(hq, hkv, d, P, 2, 600)
    for s in range(2):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(330 + s, hkv, d, s), W.normal((330 + s, hkv, d), s + 5, device="cuda"))
    x = W.normal((2, hq + 2 * hkv, d), 9, device="cuda")
    q, k, v = x[:, :hq].contiguous(), x[:, hq:hq + hkv].contiguous(), x[:, hq + hkv:].contiguous()
    p = torch.randint(0, 1000, (3, 2), device="cuda")
    of = [i % 3 for i in range(64)]
    out, lse = torch.empty_like(q), torch.empty(2, hq, device="cuda")
    pages = torch.empty(2, hkv, 7, dtype=torch.int32, device="cuda")
    qr = torch.empty_like(q)

    def step():
        c.append_kv_rope_axes(0, [0, 1], [0, 1, 2], q, k, v, p, of, pos=[329, 330], q_out=qr)
        c.decode_select(0, [0, 1], qr, 4, 1, 2, out=out, lse=lse, pages=pages)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for r in range(3):
        y = W.normal((2, hq + 2 * hkv, d), 20 + r, device="cuda")
        q.copy_(y[:, :hq]), k.copy_(y[:, hq:hq + hkv]), v.copy_(y[:, hq + hkv:])
        p.copy_(torch.randint(0, 1000, (3, 2), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), pages.clone()
        _check_select(c, [0, 1], pols, qr, 4, 1, 2, what="replay %d" % r, res=got)
    # the written tokens' page fills, then a replay writes into it
    c.append_kv(0, [0, 1], [0, 40, 80], _keys(80, hkv, d, 77), W.normal((80, hkv, d), 78, device="cuda"))
    k.copy_(W.normal((2, hkv, d), 79, device="cuda") * 3)
    g.replay()
    torch.cuda.synchronize()
    _check_bounds(c, [0, 1], [0])
    assert c.status() == 0


def test_two_graphs_and_an_eager_call_share_the_scratch():
    gpu_ready()
    hq, hkv, d, P = 16, 4, 64, 16
    pols = [W.HeadPolicy(G)] * 4
    c = _mk(hq, hkv, d, P, 3, 3000)
    for s in range(3):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(2900 - 900 * s, hkv, d, s), W.normal((2900 - 900 * s, hkv, d), s + 5, device="cuda"))
    q = W.normal((3, hq, d), 9, device="cuda")
    calls = [([0, 1, 2], 20, 1, 1), ([2, 0], 50, 0, 3), ([1], 3, 2, 2)]
    want = [c.decode_select(0, ids, q[:len(ids)].contiguous(), t, f, r) for ids, t, f, r in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for ids, t, f, r in calls[:2]:
        qq = q[:len(ids)].contiguous()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.decode_select(0, ids, qq, t, f, r))
        graphs.append((g, qq))
    for turn in range(3):
        for g, _ in graphs if turn % 2 == 0 else graphs[::-1]:
            g.replay()
        got = c.decode_select(0, [1], q[:1].contiguous(), 3, 2, 2)
        torch.cuda.synchronize()
        for a, b in zip(outs + [got], want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    assert c.status() == 0


def test_the_same_bits_every_time():
    gpu_ready()
    c = _mk(32, 8, 128, 64, 4, 9000)
    pols = [W.HeadPolicy(G)] * 8
    for s in range(4):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, _keys(8000 + 77 * s, 8, 128, s), W.normal((8000 + 77 * s, 8, 128), s + 5, device="cuda"))
    q = W.normal((4, 32, 128), 9, device="cuda")
    first = c.decode_select(0, [0, 1, 2, 3], q, 20, 1, 3)
    for _ in range(10):
        for a, b in zip(first, c.decode_select(0, [0, 1, 2, 3], q, 20, 1, 3)):
            assert torch.equal(a, b)


def test_a_serving_run():
    """As a model calls them: an image prompt rotated, prefilled and stored, then
    steps of write and decode over chosen pages."""
    import head_aware_paged_gb300 as H
    gpu_ready()
    hq, hkv, d, P, n = 8, 2, 128, 16, 500
    pols = [W.HeadPolicy(G), W.HeadPolicy(L, 4, 60)]
    c = _mk(hq, hkv, d, P, 1, 700)
    c.set_policy(0, to_c_policies([pols]))
    of = [0] * 16 + [1] * 24 + [2] * 24
    x = W.normal((n, hq + 2 * hkv, d), 1, device="cuda")
    i = torch.arange(n, device="cuda")
    pos = torch.stack([i // 100, i // 10 % 10, i % 10])
    q, k = H.sp_rope_axes(x[:, :hq], x[:, hq:hq + hkv], pos, of)
    v = x[:, hq + hkv:].contiguous()
    out, lse = c.prefill(0, [0], [0, n], q, k, v)
    rows = [0, 63, 499]
    ref = attend(q[rows].double().cpu(), k.double().cpu(), v.double().cpu(), rows, [(G, 0, 0, None), (L, 4, 60, None)])
    check(out[rows].cpu(), lse[rows].cpu(), ref, 2.0 ** -8, 0.0, "prefill")
    c.append_kv(0, [0], [0, n], k, v)
    for t in range(n, n + 17):
        y = W.normal((1, hq + 2 * hkv, d), t, device="cuda")
        at = torch.full((3, 1), 10 + t - n, device="cuda")
        qr = c.append_kv_rope_axes(0, [0], [0, 1], y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], at, of)
        _check_select(c, [0], pols, qr, 5, 1, 2, what="step %d" % t)


def test_refusals():
    import head_aware_paged_gb300 as H
    gpu_ready()
    c = _mk(8, 2, 128, 64, 2, 600, attach=False)
    pols = [W.HeadPolicy(G), W.HeadPolicy(G)]
    for s in range(2):
        c.set_policy(s, to_c_policies([pols]))
    q = W.normal((1, 8, 128), 9, device="cuda")
    k = _keys(300, 2, 128, 1)
    c.build(0, 0, k, k)
    with pytest.raises(H.SegPagedError):                       # no bounds
        c.decode_select(0, [0], q, 2)
    with pytest.raises(H.SegPagedError):                       # tokens held
        c.attach_page_bounds()
    c.release(0)
    buf = torch.empty(H.sp_page_bounds_bytes(c.cfg) + 512, dtype=torch.uint8, device="cuda")
    with pytest.raises(H.SegPagedError):
        H.sp_attach_page_bounds(c.handle, buf[(-buf.data_ptr()) % 256 + 16:])
    c.attach_page_bounds()
    with pytest.raises(H.SegPagedError):                       # an empty sequence
        c.decode_select(0, [0], q, 2)
    c.build(0, 0, k, k)
    for kw in (dict(top_pages=-1), dict(sink_pages=-1), dict(recent_pages=0), dict(top_pages=(1 << 20) + 1),
               dict(score_cap=100.0), dict(score_cap=0.001)):
        a = dict(top_pages=2)
        a.update(kw)
        with pytest.raises(H.SegPagedError):
            c.decode_select(0, [0], q, want_pages=False, **a)
    with pytest.raises(H.SegPagedError):
        c.decode_select(1, [0], q, 2)
    with pytest.raises(H.SegPagedError):
        c.decode_select(0, [0, 0], q.repeat(2, 1, 1), 2)
    for bad in (q.float(), q[:, :4], q.cpu(), q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(AssertionError):
            c.decode_select(0, [0], bad, 2)
    with pytest.raises(AssertionError):
        c.decode_select(0, [0], q, 2, pages=torch.empty(1, 2, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        c.decode_select(0, [0], q, 2, score_cap=0.0)
    c.release(0)
    H.sp_attach_page_bounds(c.handle, None)                    # detached
    c.build(0, 0, k, k)
    with pytest.raises(H.SegPagedError):
        c.decode_select(0, [0], q, 2)
    assert c.status() == 0


def test_two_caches_on_two_streams():
    """Each cache has its own bounds and scratch: calls on both may run at once."""
    gpu_ready()
    caches, want, qs = [], [], []
    pols = [W.HeadPolicy(G)] * 4
    for i, kv in enumerate(("bf16", "fp4")):
        c = _mk(16, 4, 128, 16, 2, 40000, kv=kv)
        for s in range(2):
            c.set_policy(s, to_c_policies([pols]))
            n = 38000 if s == 0 else 3000
            c.build(s, 0, _keys(n, 4, 128, 10 * i + s), W.normal((n, 4, 128), s + 5, device="cuda"))
        q = W.normal((2, 16, 128), 9 + i, device="cuda")
        caches.append(c)
        qs.append(q)
        want.append([c.decode_select(0, [0, 1], q, top, 1, 2) for top in (40, 2100)])      # one launch, two launches
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    got = [[], []]
    for _ in range(5):
        for i, c in enumerate(caches):
            for top in (40, 2100):
                with torch.cuda.stream(streams[i]):
                    got[i].append(c.decode_select(0, [0, 1], qs[i], top, 1, 2))
    torch.cuda.synchronize()
    for i in range(2):
        for k, res in enumerate(got[i]):
            for a, b in zip(res, want[i][k % 2]):
                assert torch.equal(a, b), (i, k)
        assert caches[i].status() == 0


@pytest.mark.parametrize("top", [3, 2100])
def test_stream_argument_and_launch_events(top):
    gpu_ready()
    c = _mk(4, 1, 64, 16, 1, 40000)
    c.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = _keys(39000, 1, 64, 1)
    c.build(0, 0, k, k)
    q = W.normal((1, 4, 64), 9, device="cuda")
    want = c.decode_select(0, [0], q, top)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for x in e:
        x.record(s)
    c.set_launch_events(*e)
    got = c.decode_select(0, [0], q, top, stream=s)
    s.synchronize()
    assert 0.0 < e[0].elapsed_time(e[1]) < 1000.0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_largest_batch():
    """512 sequences of 8 KV heads, a few tokens to a few pages each."""
    gpu_ready()
    hkv, P = 8, 16
    pols = [W.HeadPolicy(G) if h % 2 == 0 else W.HeadPolicy(L, 2, 9) for h in range(hkv)]
    lens = [1 + (37 * s) % 150 for s in range(512)]
    c = _mk(hkv, hkv, 64, P, 512, 160, batch=512)
    x, y = _keys(150, hkv, 64, 1), W.normal((150, hkv, 64), 2, device="cuda")
    for s, n in enumerate(lens):
        c.set_policy(s, to_c_policies([pols]))
        c.build(s, 0, x[150 - n:], y[150 - n:])
    q = W.normal((512, hkv, 64), 3, device="cuda")
    out, lse, pages = c.decode_select(0, list(range(512)), q, 2, 1, 1)
    for s in (0, 1, 4, 100, 255, 256, 511):
        _check_select(c, [s], pols, q[s:s + 1], 2, 1, 1, what=str(s), res=(out[s:s + 1], lse[s:s + 1], pages[s:s + 1]))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_pools_past_4_gib(kv):
    """The same sequence at the start of a pool and behind 4 GiB of keys: the same
    pages, the same bits."""
    gpu_ready()
    hkv, P, n = 8, 128, 262144
    per = hkv * n // P                                        # pages a filler takes
    fill = -(-(1 << 32) // (per * P * 128 * (2 if kv == "bf16" else 1)))
    k = torch.randn(n, hkv, 128, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    m = 9000
    ks, vs = _keys(m, hkv, 128, 1), W.normal((m, hkv, 128), 2, device="cuda")
    q = W.normal((1, 16, 128), 3, device="cuda")
    res = []
    for fillers in (0, fill):
        c = _mk(16, hkv, 128, P, fill + 1, n, pages=fillers * per + hkv * (m // P + 1), kv=kv)
        pol = to_c_policies([[W.HeadPolicy(G)] * hkv])
        for s in range(fillers):
            c.set_policy(s, pol)
            c.build(s, 0, k, k)
        c.set_policy(fill, pol)
        c.build(fill, 0, ks, vs)
        if fillers:
            assert min(c.export_table(fill, 0, 7)[0]) * P * 128 * (2 if kv == "bf16" else 1) >= 1 << 32
        res.append([c.decode_select(0, [fill], q, t, 1, 2) for t in (5, 60)])
        torch.cuda.synchronize()
        assert c.status() == 0
        c.close()
        del c
    for a, b in zip(*res):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("cap", [1.5, 50.0, 64.0])
def test_capped_lse_of_one_key(kv, cap):
    """One key and one product a head, so lse = cap tanh(s / cap) with nothing summed:
    s and s / cap three roundings of 2^-24, tanh two steps of 2^-23, times the cap
    and back to e one each (2^-20.5 of it in all); the weight's exp2 and the sum's
    log2 2^-22 each, absolute, with their constants' roundings 2^-20."""
    gpu_ready()
    hq = 16
    c = _mk(hq, 1, 128, 16, 1, 64, kv=kv)
    c.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = torch.zeros(1, 1, 128, device="cuda", dtype=torch.bfloat16)
    k[0, 0, 77] = 1.5                                           # exact in every page type
    c.build(0, 0, k, k)
    q = torch.zeros(1, hq, 128, device="cuda", dtype=torch.bfloat16)
    q[0, :, 77] = torch.tensor([0.0, 1e-4, -1e-3, 0.01, 0.1, -0.5, 1.0, 3.0, -7.0, 20.0, 60.0, -150.0, 300.0, 900.0, -2000.0, 1e4])
    out, lse, _ = c.decode_select(0, [0], q, 1, score_cap=cap)
    s = q[0, :, 77].double().cpu() * 1.5 / np.sqrt(128.0)
    want = cap * torch.tanh(s / cap)
    err = (lse[0].double().cpu() - want).abs()
    assert (err <= 2.0 ** -20.5 * want.abs() + 2.0 ** -20).all(), (err / (2.0 ** -20.5 * want.abs() + 2.0 ** -20)).max()
    assert torch.equal(out[0, :, 77].cpu(), torch.full((hq,), 1.5, dtype=torch.bfloat16))
