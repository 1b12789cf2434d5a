"""GPU: attention over scores capped by cap * tanh(s / cap), prefill and
decode, every page type, against 64 bits.

Tolerances count roundings (tests/_attn64.py): prefill rounds P to bf16
(2^-8 of each weight), decode to bf16 (bf16 pages) or f16 (FP8 and 4-bit
pages, 2^-11, whose query times channel scale is f16 too, 2^-11 of each
product); prefill reads FP8 rows rounded to bf16 (2^-8 of K's and V's).  The
cap only shrinks what a score may be off by."""
import math

import numpy as np
import pytest
import torch

import workloads as W
from _attn64 import attend, check
from _gpu_common import f64, gpu_ready, pol_tuple, to_c_policies
from oracle import fp4, fp8

pytestmark = pytest.mark.gpu

G, L, R = W.GLOBAL, W.LOCAL, W.RETRIEVAL


def _mk(hq, hkv, d, P, seqs, max_len, pages, kv="bf16"):
    import head_aware_paged_gb300 as H
    return H.SegPagedCache(H.Config(num_layers=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P,
                                    max_seqs=seqs, max_seq_len=max_len, num_pages=pages, max_idx_per_seq=8192,
                                    max_tokens=max_len, max_batch=seqs,
                                    kv_dtype={"bf16": H.KV_BF16, "fp8": H.KV_FP8, "fp4": H.KV_FP4}[kv]))


def _held(x, kv, s):
    """What the pages hold of rows x [n, hkv, d], 64 bits on the device."""
    if kv == "bf16" or x.shape[0] == 0:
        return x.double()
    xs = f64(x)
    f = (lambda y, h: fp8.dequantize(fp8.quantize(y, s[h]), s[h])) if kv == "fp8" else (lambda y, h: fp4.stored(y))
    return torch.tensor(np.stack([f(xs[:, h], h) for h in range(xs.shape[1])], 1), device="cuda")


def _pols(hkv, n):
    idx = np.arange(min(n, 70), n, 3, dtype=np.int32)          # early rows see nothing
    return [W.HeadPolicy(G), W.HeadPolicy(L, 4, 90), W.HeadPolicy(R, idx=idx), W.HeadPolicy(L, 0, 1)][:hkv]


CASES = [("bf16", 64, 16, 6, 2), ("bf16", 64, 128, 4, 4), ("bf16", 128, 64, 32, 4), ("bf16", 128, 32, 3, 3),
         ("fp8", 128, 64, 16, 4), ("fp8", 128, 16, 3, 1), ("fp4", 128, 32, 8, 4), ("fp4", 128, 128, 36, 3)]


@pytest.mark.parametrize("cap,qs", [(50.0, 1.0), (30.0, 12.0), (2.0, 1.0), (1.0 / 64, 3.0), (64.0, 40.0)])
@pytest.mark.parametrize("kv,d,P,hq,hkv", CASES)
def test_prefill_and_decode(kv, d, P, hq, hkv, cap, qs):
    """qs spreads the scores: well inside the cap, around it, far past it."""
    gpu_ready()
    n, c = 300, 141
    cache = _mk(hq, hkv, d, P, 2, n + c, 2 * hkv * ((n + c) // P + 4), kv)
    pols = _pols(hkv, n + c)
    pt = [pol_tuple(p) for p in pols]
    ks = np.full((hkv, d), 2.0 ** -6, np.float32)
    for s in range(2):
        if kv == "fp8" and s == 0:
            cache.set_kv_scales(0, ks, ks)
        cache.set_policy(s, to_c_policies([pols]))
    hist = [W.normal((n, hkv, d), 5 + i, device="cuda") for i in range(2)]
    cache.build(0, 0, *hist)                                   # sequence 1 starts empty
    q = (W.normal((2 * c, hq, d), 7, device="cuda").float() * qs).to(torch.bfloat16)
    k, v = W.normal((2 * c, hkv, d), 8, device="cuda"), W.normal((2 * c, hkv, d), 9, device="cuda")
    out, lse = cache.prefill(0, [0, 1], [0, c, 2 * c], q, k, v, score_cap=cap)
    hk, hv = _held(hist[0], kv, ks), _held(hist[1], kv, ks)
    for b, m in ((0, n), (1, 0)):
        sl = slice(b * c, b * c + c)
        ref = attend(q[sl].double(), torch.cat([hk[:m], k[sl].double()]), torch.cat([hv[:m], v[sl].double()]),
                     range(m, m + c), pt, cap)
        check(out[sl], lse[sl], ref, 2.0 ** -8, 0.0, "prefill %d" % b, cap)
    cache.append_kv(0, [0, 1], [0, c, 2 * c], k, v)
    qd = q[[c - 1, 2 * c - 1]].contiguous()
    out, lse = cache.decode(0, [0, 1], qd, score_cap=cap)
    for b, m in ((0, n), (1, 0)):
        sl = slice(b * c, b * c + c)
        kk = torch.cat([hk[:m], _held(k[sl], kv, ks)])
        vv = torch.cat([hv[:m], _held(v[sl], kv, ks)])
        ref = attend(qd[b:b + 1].double(), kk, vv, [m + c - 1], pt, cap)
        # q * scale is exact in f16 (a power of two), so scores carry no rounding
        check(out[b:b + 1], lse[b:b + 1], ref, 2.0 ** -8 if kv == "bf16" else 2.0 ** -11, 0.0, "decode %d" % b, cap)
    assert cache.status() == 0


def test_long_split_items():
    """A chunk of two row blocks over a long history: items in pieces, merged."""
    gpu_ready()
    hq, hkv, d, P, n, c, cap = 4, 2, 128, 64, 20000, 140, 30.0
    cache = _mk(hq, hkv, d, P, 1, n + c, 2 * hkv * ((n + c) // P + 4))
    pols = [W.HeadPolicy(G), W.HeadPolicy(L, 4, 9000)]
    cache.set_policy(0, to_c_policies([pols]))
    hist = [W.normal((n, hkv, d), 5 + i, device="cuda") for i in range(2)]
    cache.build(0, 0, *hist)
    q = (W.normal((c, hq, d), 7, device="cuda").float() * 8).to(torch.bfloat16)
    k, v = W.normal((c, hkv, d), 8, device="cuda"), W.normal((c, hkv, d), 9, device="cuda")
    out, lse = cache.prefill(0, [0], [0, c], q, k, v, score_cap=cap)
    rows = [0, 1, 77, 127, 128, c - 1]
    ref = attend(q[rows].double(), torch.cat([hist[0], k]).double(), torch.cat([hist[1], v]).double(),
                 [n + r for r in rows], [pol_tuple(p) for p in pols], cap)
    check(out[rows], lse[rows], ref, 2.0 ** -8, 0.0, "split", cap)
    assert cache.status() == 0


@pytest.mark.parametrize("cap", [1.0 / 64, 1.0, 50.0, 64.0])
def test_extreme_scores(cap):
    """Scores of +-1e30 and rows all at -cap: weights at the ends of the
    exponentials' range, equal where every score sits on the cap."""
    gpu_ready()
    d, n = 64, 200
    cache = _mk(1, 1, d, 16, 1, n, 20)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = torch.full((n, 1, d), 1e15, dtype=torch.bfloat16, device="cuda")
    k[1::2] *= -1
    q = torch.full((n, 1, d), 1e15, dtype=torch.bfloat16, device="cuda")
    q[100:] *= -1
    k[:, :, 1:], q[:, :, 1:] = 0, 0
    v = W.normal((n, 1, d), 3, device="cuda")
    out, lse = cache.prefill(0, [0], [0, n], q, k, v, score_cap=cap)
    ref = attend(q.double(), k.double(), v.double(), range(n), [(G, 0, 0, None)], cap)
    ref = ref[:3] + (torch.zeros_like(ref[3]), ref[4])         # every score is +-cap, exactly
    check(out, lse, ref, 2.0 ** -8, 0.0, "prefill", cap)
    low = torch.full_like(k, -1e15)                             # every score at -cap
    low[:, :, 1:] = 0
    q[:] = q[:1].abs()
    out, lse = cache.prefill(0, [0], [0, n], q, low, v, score_cap=cap)
    ref = attend(q.double(), low.double(), v.double(), range(n), [(G, 0, 0, None)], cap)
    check(out, lse, ref[:3] + (torch.zeros_like(ref[3]), ref[4]), 2.0 ** -8, 0.0, "all low", cap)
    cache.append_kv(0, [0], [0, n], low, v)
    out, lse = cache.decode(0, [0], q[:1].contiguous(), score_cap=cap)
    mean = v.double().mean(0, keepdim=True)
    assert ((out.double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -8 * v.double().abs().mean(0)).all()
    assert abs(lse.item() - (math.log(n) - cap)) <= 2.0 ** -18 * (1 + cap) + 3e-7 * cap
    assert cache.status() == 0


@pytest.mark.parametrize("cap", [1.0 / 64, 1.0, 50.0, 64.0])
@pytest.mark.parametrize("d", [64, 128])
def test_extreme_scores_decode(d, cap):
    """Scores of +-1e30, both signs of the query: every score sits on +-cap."""
    gpu_ready()
    n = 200
    cache = _mk(2, 1, d, 16, 1, n, 20)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    k[:, :, 0] = 1e15
    k[1::3] *= -1
    v = W.normal((n, 1, d), 3, device="cuda")
    cache.append_kv(0, [0], [0, n], k, v)
    q = torch.zeros(1, 2, d, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0], q[:, 1, 0] = 1e15, -1e15
    out, lse = cache.decode(0, [0], q, score_cap=cap)
    ref = attend(q.double(), k.double(), v.double(), [n - 1], [(G, 0, 0, None)], cap)
    check(out, lse, ref[:3] + (torch.zeros_like(ref[3]), ref[4]), 2.0 ** -8, 0.0, "decode", cap)
    assert cache.status() == 0


@pytest.mark.parametrize("cap", [0.5, 1.0, 50.0, 64.0])
@pytest.mark.parametrize("d", [64, 128])
def test_cap_pointwise(d, cap):
    """Each row sees one key, so lse is the capped score itself: every warp of
    32 rows stays below another multiple of the cap.  The score is one product
    (exact) times 1 / sqrt(d).  Tolerance: 1.3e-7 cap of the approximation;
    fp32 roundings, in log2 units, of the reference ref and of sums up to ref
    + 2 a (a = cap log2 e, 2^-24 each, 16 of them); 2^-21 of exp2 and log2."""
    gpu_ready()
    tops = [0.02, 0.1, 0.11, 0.2, 0.27, 0.29, 0.45, 0.52, 0.8, 1.5, 4.0, 30.0]
    n = 32 * len(tops)
    cache = _mk(1, 1, d, 16, 1, n, 40)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(L, 0, 1)]]))
    y = torch.cat([torch.linspace(-t, t, 32, dtype=torch.float64) for t in tops])
    q = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros_like(q)
    q[:, 0, 1] = (y * cap * math.sqrt(d) / 3).to(torch.bfloat16).cuda()
    k[:, 0, 1] = 3.0
    v = W.normal((n, 1, d), 3, device="cuda")
    out, lse = cache.prefill(0, [0], [0, n], q, k, v, score_cap=cap)
    want = cap * torch.tanh(q[:, 0, 1].double() * 3 / math.sqrt(d) / cap)
    a = cap * math.log2(math.e)
    tol = 1.3e-7 * cap + 16 * 2.0 ** -24 * (abs(118 - a) if 118 - a < a else a) + 32 * 2.0 ** -24 * a + 2.0 ** -21
    worst = ((lse[:, 0].double() - want).abs() / tol).max().item()
    assert worst <= 1.0, worst
    # one weight: P / l is 1 but for P's rounding to bf16, then the output's
    assert ((out.double() - v.double()).abs() <= 2.0 ** -7 * 1.01 * v.double().abs()).all()
    assert cache.status() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("cap,qs", [(50.0, 1.0), (2.0, 12.0)])
def test_nan_query_stays_in_its_row(kv, cap, qs):
    """A NaN query answers NaN, inside the cap and far past it, and the
    other rows of its tile stay right."""
    gpu_ready()
    hq, d, n = 2, 128, 200
    cache = _mk(hq, 1, d, 64, 1, n, 10, kv)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    q = (W.normal((n, hq, d), 7, device="cuda").float() * qs).to(torch.bfloat16)
    k, v = W.normal((n, 1, d), 8, device="cuda"), W.normal((n, 1, d), 9, device="cuda")
    want, want_lse = cache.prefill(0, [0], [0, n], q, k, v, score_cap=cap)
    bad = q.clone()
    bad[[5, 150], 1, 3] = math.nan
    got, lse = cache.prefill(0, [0], [0, n], bad, k, v, score_cap=cap)
    hit = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    hit[[5, 150], 1] = True
    assert torch.isnan(got[hit]).all()
    ref = attend(q.double(), k.double(), v.double(), range(n), [(G, 0, 0, None)], cap)
    got[hit], lse[hit] = want[hit], want_lse[hit]               # (checked above)
    check(got, lse, ref, 2.0 ** -8, 0.0, "the other rows", cap)
    cache.append_kv(0, [0], [0, n], k, v)
    got, _ = cache.decode(0, [0], bad[150:151].contiguous(), score_cap=cap)
    assert torch.isnan(got[0, 1]).all() and torch.isfinite(got[0, 0]).all()
    assert cache.status() == 0


def test_uncapped_calls_keep_their_results_and_refusals():
    gpu_ready()
    from head_aware_paged_gb300 import SegPagedError
    cache = _mk(4, 2, 64, 16, 1, 128, 40)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)] * 2]))
    q, k, v = (W.normal((50, h, 64), 1 + h, device="cuda") for h in (4, 2, 2))
    a = cache.prefill(0, [0], [0, 50], q, k, v)
    cache.prefill(0, [0], [0, 50], q, k, v, score_cap=5.0)
    b = cache.prefill(0, [0], [0, 50], q, k, v)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cache.append_kv(0, [0], [0, 50], k, v)
    for cap in (0.0, -1.0, 1.0 / 65, 64.5, math.inf, math.nan):
        with pytest.raises(SegPagedError):
            cache.prefill(0, [0], [0, 50], q, k, v, score_cap=cap)
        with pytest.raises(SegPagedError):
            cache.decode(0, [0], q[:1].contiguous(), score_cap=cap)
    assert cache.status() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("hist", [0, 7000])
@pytest.mark.parametrize("cap", [None, 50.0, 2.0])
def test_nan_query_has_a_nan_lse(cap, hist, kv):
    """-inf says that a row saw nothing; a NaN row saw something.  Over a long
    history the items are split and merged."""
    gpu_ready()
    hq, d, n = 2, 128, 140
    cache = _mk(hq, 1, d, 64, 1, hist + n, (hist + n) // 64 + 4, kv)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(R, idx=np.arange(3, hist + n, dtype=np.int32))]]))
    if hist:
        cache.build(0, 0, *(W.normal((hist, 1, d), 5 + i, device="cuda") for i in range(2)))
    q, k, v = (W.normal((n, h, d), 7 + h, device="cuda") for h in (hq, 1, 1))
    q[[5, 130], 1, 3] = math.nan
    out, lse = cache.prefill(0, [0], [0, n], q, k, v, score_cap=cap)
    hit = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    hit[[5, 130], 1] = True
    none = torch.zeros_like(hit)
    none[:max(0, 3 - hist)] = True
    assert torch.equal(torch.isnan(lse), hit) and torch.equal(torch.isneginf(lse), none)
    assert torch.equal(torch.isnan(out).all(-1), hit) and torch.equal(torch.isnan(out).any(-1), hit)
    assert (out[none] == 0).all()
    cache.append_kv(0, [0], [0, n], k, v)
    out, lse = cache.decode(0, [0], q[130:131].contiguous(), score_cap=cap)
    assert torch.isnan(lse[0]).tolist() == [False, True] and torch.isnan(out[0, 1]).all()
    assert cache.status() == 0


@pytest.mark.parametrize("cap", [1.0, 30.0, 50.0, 64.0])
@pytest.mark.parametrize("sign,vs", [(-1, 2.0 ** -28), (-1, 2.0 ** 18), (1, 2.0 ** -28), (1, 2.0 ** 18)])
@pytest.mark.parametrize("d,hq", [(64, 1), (128, 2)])
def test_small_and_large_values(d, hq, sign, vs, cap):
    """Every score at -cap or at +cap, values around 2^-28 and 2^18: what weight
    times value sums to stays inside fp32's normal range."""
    gpu_ready()
    n = 300
    cache = _mk(hq, 1, d, 16, 1, 2 * n, 60)
    cache.set_policy(0, to_c_policies([[W.HeadPolicy(G)]]))
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    k[:, :, 0] = 1e15
    q = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = sign * 1e15
    v = (W.normal((n, 1, d), 3, device="cuda").float() * vs).to(torch.bfloat16)

    def held(rows, keys, values):
        ref = attend(q[:len(rows)].double(), keys.double(), values.double(), rows, [(G, 0, 0, None)], cap)
        return ref[:3] + (torch.zeros_like(ref[3]), ref[4])    # every score is +-cap, exactly

    out, lse = cache.prefill(0, [0], [0, n], q, k, v, score_cap=cap)
    check(out, lse, held(range(n), k, v), 2.0 ** -8, 0.0, "prefill", cap)
    cache.append_kv(0, [0], [0, n], k, v)
    out, lse = cache.prefill(0, [0], [0, n], q, k, v, score_cap=cap)          # over history too
    check(out, lse, held(range(n, 2 * n), torch.cat([k, k]), torch.cat([v, v])), 2.0 ** -8, 0.0, "history", cap)
    out, lse = cache.decode(0, [0], q[:1].contiguous(), score_cap=cap)
    check(out, lse, held([n - 1], k, v), 2.0 ** -8, 0.0, "decode", cap)
    assert cache.status() == 0


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("kv,d,hq,hkv", [("bf16", 64, 6, 3), ("bf16", 64, 4, 2), ("bf16", 128, 3, 3), ("bf16", 128, 8, 2),
                                         ("fp8", 128, 8, 2), ("fp8", 128, 3, 3), ("fp4", 128, 3, 3), ("fp4", 128, 8, 2)])
def test_every_page_size(kv, d, hq, hkv, P):
    """Each instance at each page size: history that ends inside a page, rings
    that wrap inside a tile."""
    gpu_ready()
    n, c, cap = 333, 70, 20.0
    cache = _mk(hq, hkv, d, P, 1, n + c, hkv * ((n + c) // P + 4), kv)
    pols = _pols(hkv, n + c)
    pt = [pol_tuple(p) for p in pols]
    ks = np.full((hkv, d), 2.0 ** -6, np.float32)
    if kv == "fp8":
        cache.set_kv_scales(0, ks, ks)
    cache.set_policy(0, to_c_policies([pols]))
    hist = [W.normal((n, hkv, d), 5 + i, device="cuda") for i in range(2)]
    cache.build(0, 0, *hist)
    q, k, v = (W.normal((c, h, d), 7 + i, device="cuda") for i, h in enumerate((hq, hkv, hkv)))
    hk, hv = _held(hist[0], kv, ks), _held(hist[1], kv, ks)
    out, lse = cache.prefill(0, [0], [0, c], q, k, v, score_cap=cap)
    ref = attend(q.double(), torch.cat([hk, k.double()]), torch.cat([hv, v.double()]), range(n, n + c), pt, cap)
    check(out, lse, ref, 2.0 ** -8, 0.0, "prefill", cap)
    out, lse = cache.decode(0, [0], q[:1].contiguous(), score_cap=cap)
    check(out, lse, attend(q[:1].double(), hk, hv, [n - 1], pt, cap), 2.0 ** -8 if kv == "bf16" else 2.0 ** -11, 0.0, "decode", cap)
    assert cache.status() == 0
