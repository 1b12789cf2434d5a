"""Performance cases of the rotation with several axes and of the decode over chosen pages.

Two operators, in the calls that serve a model:

  rotate  `sp_rope_axes`: a prompt chunk's queries and keys rotated to their positions
          on several axes (time, height, width), before its prefill
  write   `append_kv_rope_axes`: new queries and keys rotated so, the rotated keys and
          the values written into their heads' pages
  decode  `decode_select`: one query a sequence; a GLOBAL head reads its first and its
          newest pages and those whose bounds promise the largest scores
  prompt  a request's life: prompts written, their first tokens decoded, released

`run` computes them with elementary torch operations (own = False) or with the
package (own = True).  KV heads 0 .. globals-1 are GLOBAL, the others see their `sink`
first tokens and the newest `window`.

A page's bounds are the largest and the smallest of its stored keys in every
dimension, in steps of a power of two: the least 2^e, -50 <= e <= 50, that takes the
page's largest magnitude to at most 127; the upper bound rounded up, the lower one
down.  A query head is rounded to such steps of its own.  A page's score for a head is
sum_c max(x_c hi_c, x_c lo_c), times both steps, and the largest of the KV head's query
heads counts.  Kept are the first `first` and the newest `newest` pages and the `top`
others with the highest scores, ties to the lower page.

4-bit pages: 16 neighbouring dimensions share a scale with 5 exponent and 3 mantissa
bits, the value nearest amax / 6 (ties to even, at most 10240); an element is the e2m1
value (0, .5, 1, 1.5, 2, 3, 4, 6, signed) nearest x / scale (ties to an even mantissa).
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ROW_BYTES = {"bf16": 2.0, "fp8": 1.0, "fp4": 0.5625}     # per element, scales included


def listed():
    """A head layout of 32 query and 8 KV heads, one GLOBAL head of eight (or all), sink 4,
    windows of 1024 to 2048 and page 64 are the repository's own."""
    base = dict(hq=32, hkv=8, d=128, page=64, globals=1, sink=4, window=1024, ragged=False, mixed=False)
    wr = dict(base, kind="write", pages="bf16", theta=500000.0)
    rot = dict(base, kind="rotate", theta=500000.0)
    dec = dict(base, kind="decode", pages="bf16", cap=0.0, globals=8, first=1, newest=7, top=24)
    return [
        # the new token of each of 64 sequences in a serving step: latency
        dict(wr, name="write_axes_step_64", seqs=64, hist=500, new=1),
        # a whole prompt of text and frames written after its projections
        dict(wr, name="write_axes_prompt_8k", seqs=1, hist=0, new=8192),
        # several short prompts of odd lengths, a small model's heads, axes mixed pair by pair
        dict(wr, name="write_axes_ragged_d64", seqs=7, hist=90, new=333, theta=10000.0, hq=14, hkv=2, d=64, page=16,
             window=100, ragged=True, mixed=True),
        # one image and its question, before prefill
        dict(rot, name="rotate_axes_777", seqs=1, new=777, hq=28, hkv=4, mixed=True),
        # the largest chunk: a video's prompt
        dict(rot, name="rotate_axes_32k", seqs=1, new=32768),
        # one user's conversation, few pages: the smallest step
        dict(dec, name="select_single_4k", seqs=1, hist=4095, first=1, newest=2, top=13),
        # one long document, a quarter of the heads GLOBAL
        dict(dec, name="select_single_128k", seqs=1, hist=131072, globals=2, window=2048, newest=4, top=123),
        # 32 sequences of 32K tokens, every head GLOBAL, a sixteenth of the pages read
        dict(dec, name="select_32x32k", seqs=32, hist=32768),
        # FP8 pages, odd lengths, an odd group of query heads
        dict(dec, name="select_fp8_ragged", pages="fp8", seqs=9, hist=20001, hq=35, hkv=5, globals=3, page=32, window=1500,
             first=2, newest=5, top=57, ragged=True),
        # 4-bit pages, every head GLOBAL
        dict(dec, name="select_fp4_16x32k", pages="fp4", seqs=16, hist=32768),
        # capped scores, small pages, one query head a KV head
        dict(dec, name="select_cap_d64", cap=30.0, seqs=6, hist=7001, hq=12, hkv=12, d=64, page=16, globals=5, window=300,
             first=0, newest=1, top=40, ragged=True),
        # four prompts stored, their first tokens decoded, released
        dict(dec, name="prompt_4x8k", kind="prompt", seqs=4, hist=8192),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rotate", "write", "decode", "decode", "decode", "prompt"])
    pages = rng.choice(["bf16", "fp8", "fp4"]) if kind in ("decode", "prompt") else "bf16"
    d = 128 if pages != "bf16" else rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8])
    c = dict(kind=kind, pages=pages, d=d, hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 4, 7, 8, 12]),
             page=rng.choice([16, 32, 64, 64, 128]), globals=rng.randint(0, hkv), sink=rng.choice([0, 4, 4, 37]),
             window=_log(rng, 1, 4096), ragged=rng.random() < 0.6)
    if kind in ("rotate", "write"):
        c.update(theta=rng.choice([10000.0, 500000.0, 1000000.0]), mixed=rng.random() < 0.5)
        if kind == "rotate":
            c.update(seqs=1, new=_log(rng, 1, 16384))
        elif rng.random() < 0.5:
            c.update(seqs=_log(rng, 1, 128), hist=_log(rng, 1, 600), new=1)
        else:
            c.update(seqs=rng.randint(1, 4), hist=_log(rng, 1, 300), new=_log(rng, 2, 2048))
        return c
    c.update(globals=rng.randint(1, hkv), cap=rng.choice([0.0, 0.0, 1.5, 30.0, 50.0]), first=rng.choice([0, 1, 1, 3]),
             newest=_log(rng, 1, 16), top=rng.choice([0, _log(rng, 1, 200), _log(rng, 1, 200)]))
    c.update(seqs=_log(rng, 1, 32 if kind == "decode" else 3), hist=_log(rng, 1, 32767 if kind == "decode" else 8191))
    return c


# ----------------------------------------------------------- shapes and layout

def _lengths(case):
    """Tokens held before the new ones, and new tokens, of each sequence."""
    r = random.Random("%d %d" % (case["seqs"], case.get("hist", 0)))
    f = [1.0 if not case["ragged"] else math.exp(r.uniform(-1.5, 0.0)) for _ in range(case["seqs"])]
    if case["kind"] in ("decode", "prompt"):
        return [max(1, int(case["hist"] * x)) for x in f], [0] * case["seqs"]
    return [int(case.get("hist", 0) * x) for x in f], [max(1, int(case["new"] * x)) for x in reversed(f)]


def _held(case):
    return [a + b for a, b in zip(*_lengths(case))]


def _unit(case, h, n):
    """(pages, LOCAL?, sink pages, ring slots) of KV head h that holds n tokens."""
    P = case["page"]
    if h < case["globals"]:
        return -(-n // P), False, 0, 0
    ring = -(-case["window"] // P) + 1
    s = case["sink"]
    return -(-min(n, s) // P) + min(ring, -(-max(0, n - s) // P)), True, -(-s // P), ring * P


def _layout(case):
    """First page of every (sequence, KV head), and all pages: a fresh cache gives them in this order."""
    first, total = [], 0
    for n in _held(case):
        for h in range(case["hkv"]):
            first.append(total)
            total += _unit(case, h, n)[0]
    return first, total


def _slots(case, h, pos, n):
    """Slot of each position in its unit that holds n tokens, and whether it is kept."""
    _, local, sink_pages, ring = _unit(case, h, n)
    if not local:
        return pos, pos < n
    s = case["sink"]
    slot = torch.where(pos < s, pos, sink_pages * case["page"] + (pos - s).clamp(min=0) % ring)
    return slot, (pos < n) & ((pos < s) | (pos >= n - ring))


def work(case):
    hist, new = _lengths(case)
    hq, hkv, d, P, kind = case["hq"], case["hkv"], case["d"], case["page"], case["kind"]
    g, row = hq // hkv, 2 * d * ROW_BYTES[case.get("pages", "bf16")]
    byt = flo = 0.0
    if kind == "rotate":
        c = sum(new)
        return {"bytes": c * ((hq + hkv) * 4 * d + 24), "flops": 3 * d * c * (hq + hkv)}
    for a, c, n in zip(hist, new, _held(case)):
        byt += 24 * c
        for h in range(hkv):
            _, local, _, ring = _unit(case, h, n)
            kept = n if not local else min(n, case["sink"]) + min(max(0, n - case["sink"]), ring)
            if kind == "write":
                kept = c if not local else sum(1 for p in range(a, n) if p < case["sink"] or p >= n - ring)
                byt += kept * (4 * d + row) + c * g * 4 * d
                flo += 3 * d * (kept + c * g)
                continue
            seen = min(n, case["sink"] + case["window"])
            if not local:
                nb, some = -(-n // P), case["first"] + case["newest"] + case["top"]
                seen = n - max(0, nb - some) * P
                if nb > some and case["top"]:
                    cand = nb - case["first"] - case["newest"]
                    byt += cand * (2 * d + 4)
                    flo += cand * 2 * d * g
                if kind == "prompt":
                    byt += n // P * (2 * d + 4)
                    flo += 2 * d * n
            byt += seen * row + g * (4 * d + 4)
            flo += 4 * d * g * seen
            if kind == "prompt":
                byt += kept * (4 * d + row)
    return {"bytes": byt, "flops": flo}


# -------------------------------------------------------------------- inputs

def _axis_of(case):
    """The axis of each pair of dimensions: three sections (a quarter, three eighths,
    three eighths of the pairs), or the axes in turn."""
    m = case["d"] // 2
    if case["mixed"]:
        return [i % 3 for i in range(m)]
    return [0] * (m // 4) + [1] * (m // 8 * 3) + [2] * (m // 8 * 3)


def _axis_pos(case, seed):
    """Positions [3, rows]: runs of text, which move on all axes alike, and grids of
    patches (frames of a video repeat the grid); a sequence's first new token follows its history."""
    r = random.Random(seed)
    hist, new = _lengths(case)
    cols = []
    for a, c in zip(hist, new):
        at, left = a + r.randint(0, 100000), c
        while left:
            if c == 1 or r.random() < 0.5:
                n = min(left, r.randint(1, 200))
                t = torch.arange(at, at + n)
                cols.append(torch.stack([t, t, t]))
                at += n
            else:
                gh, gw, gt = r.randint(2, 40), r.randint(2, 40), r.choice([1, 1, 8])
                n = min(left, gh * gw * gt)
                i = torch.arange(n)
                cols.append(torch.stack([at + i // (gh * gw), at + i // gw % gh, at + i % gw]))
                at += max(gh, gw, gt)
            left -= n
    return torch.cat(cols, 1).to(DEV)


def _inputs(case, seed):
    """The new tokens' projections as one packed tensor, as a fused projection leaves them
    (decode: the queries), and a generator of each sequence's history.  Keys have a few
    strong channels and a direction of their own every few pages."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows = sum(_lengths(case)[1]) or case["seqs"]
    strong = torch.ones(hkv, d, device=DEV)
    strong[:, torch.randperm(d, generator=g, device=DEV)[:4]] = 6.0
    qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g, device=DEV)
    qkv[:, :hq] *= 2.0 if case.get("cap") else 1.0
    qkv[:, hq:hq + hkv] *= 0.5 * strong
    qkv = qkv.to(torch.bfloat16)

    def history():
        for n in _held(case):
            k = torch.randn(n, hkv, d, generator=g, device=DEV)
            k += torch.randn(n // 100 + 1, hkv, d, generator=g, device=DEV).repeat_interleave(100, 0)[:n]
            k = (k * (0.4 * strong)).to(torch.bfloat16)
            yield k, torch.randn(n, hkv, d, generator=g, device=DEV).to(torch.bfloat16)

    # FP8 channel scales: powers of two, as a calibration rounds them
    ex = torch.randint(-6, -2, (2, hkv, d), generator=g, device=DEV).float()
    return qkv, history, torch.exp2(ex)


def prepare(case, seed):
    qkv, history, scales = _inputs(case, seed)
    hq, hkv, d, P, kind = case["hq"], case["hkv"], case["d"], case["page"], case["kind"]
    hist, new = _lengths(case)
    held = _held(case)
    st = dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
    if kind in ("rotate", "write"):
        half = torch.arange(d // 2, dtype=torch.float64)
        st.update(axis_pos=_axis_pos(case, seed), axis_of=_axis_of(case),
                  freq=(case["theta"] ** (-2.0 * half / d)).to(DEV))
    if kind == "rotate":
        return st
    cu = [0]
    for c in new:
        cu.append(cu[-1] + c)
    st.update(cu=cu, start=list(hist), ids=list(range(case["seqs"])))
    if kind != "write":
        st["q"] = st["q"].contiguous()
    first, total = _layout(case)
    if own:
        from head_aware_paged_gb300 import GLOBAL, KV_BF16, KV_FP4, KV_FP8, LOCAL, Config, Policy, SegPagedCache
        cache = SegPagedCache(Config(
            num_layers=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P, max_seqs=case["seqs"],
            max_seq_len=max(held + [case["window"], case["sink"]]) + 1, num_pages=max(1, total),
            max_tokens=max(max(held), cu[-1]), max_batch=case["seqs"],
            kv_dtype={"bf16": KV_BF16, "fp8": KV_FP8, "fp4": KV_FP4}[case["pages"]]))
        if kind != "write":
            cache.attach_page_bounds()
        if case["pages"] == "fp8":
            cache.set_kv_scales(0, scales[0].cpu().numpy(), scales[1].cpu().numpy())
        row = [Policy(GLOBAL) if h < case["globals"] else Policy(LOCAL, case["sink"], case["window"]) for h in range(hkv)]
        prompts = []
        for b, (k, v) in enumerate(history()):
            cache.set_policy(b, [row])
            if kind == "prompt":
                prompts.append((k, v))
            else:
                cache.build(b, 0, k, v)
        st.update(cache=cache, prompts=prompts)
        return st
    # the plain form's pools, in the same page order
    rows = max(1, total) * P
    if case["pages"] == "fp4":
        pool = [torch.zeros(rows, d // 2, dtype=torch.uint8, device=DEV) for _ in range(2)]
        pool += [torch.zeros(rows, d // 16, dtype=torch.uint8, device=DEV) for _ in range(2)]
    else:
        t = torch.bfloat16 if case["pages"] == "bf16" else torch.float8_e4m3fn
        pool = [torch.zeros(rows, d, device=DEV).to(t) for _ in range(2)]
    st.update(pool=pool, scales=scales)
    n = torch.tensor(held, device=DEV)
    G = case["globals"]
    if kind != "write":
        st["page0"] = torch.tensor(first, device=DEV).view(case["seqs"], hkv)
        st["held"] = n
        st["pages"] = -(-max(held) // P)
        st["bounds"] = torch.zeros(2, max(1, total), d, device=DEV), torch.zeros(max(1, total), device=DEV)
        st["full"] = torch.cat([first[b * hkv + h] + torch.arange(held[b] // P, device=DEV)
                                for b in range(case["seqs"]) for h in range(G)] or [n[:0]])
        st["full_head"] = torch.cat([torch.full((held[b] // P,), h, device=DEV)
                                     for b in range(case["seqs"]) for h in range(G)] or [n[:0]])
    dst, src, prompts = [], [], []
    span = max([1] + held)
    where = torch.zeros(case["seqs"], hkv, span, dtype=torch.int64, device=DEV)
    for b, (k, v) in enumerate(history()):
        p = torch.arange(held[b], device=DEV)
        at_b, kept_b = [], []
        for h in range(hkv):
            slot, kept = _slots(case, h, p, held[b])
            at = first[b * hkv + h] * P + slot
            at_b.append(at[kept])
            kept_b.append(torch.stack([p[kept], torch.full_like(p[kept], h)]))
            where[b, h, :held[b]] = torch.where(kept, at, 0)
            if kind == "write":
                w = torch.arange(hist[b], held[b], device=DEV)
                w = w[kept[hist[b]:]]
                dst.append(at[w])
                src.append(torch.stack([cu[b] + w - hist[b], torch.full_like(w, h)]))
        if kind == "prompt":
            prompts.append((k, v, torch.cat(at_b), torch.cat(kept_b, 1)))
        else:
            for h in range(hkv):
                _store(st, at_b[h], k[kept_b[h][0], h], v[kept_b[h][0], h], torch.tensor(h, device=DEV))
    if kind == "write":
        st["dst"], st["src"] = torch.cat(dst), torch.cat(src, 1)
        return st
    st["prompts"] = prompts
    if kind == "decode":
        _bound(st)
    # the keys that a LOCAL unit's query sees
    s, w = case["sink"], case["window"]
    lo = (n[:, None] - w).clamp(min=s)
    lp = torch.cat([torch.arange(s, device=DEV).expand(case["seqs"], s), lo + torch.arange(w, device=DEV)], 1)
    lp = lp[:, :max(1, min(s + w, span + s))]
    st["seen"] = lp < n[:, None]
    st["at"] = torch.gather(where[:, G:], 2, lp[:, None].clamp(max=span - 1).expand(-1, hkv - G, -1))
    return st


# --------------------------------------------------------------- plain forms

def _quant4(x):
    """e2m1 codes (two a byte, the even dimension low) and scale codes of x [..., d], in
    64 bits: what lies next to a border decides a code."""
    b = x.double().unflatten(-1, (-1, 16))
    f = (b.abs().amax(-1) / 6.0).clamp(max=10240.0)
    step = torch.exp2((torch.frexp(f)[1] - 4).clamp(min=-17).double())
    scale = torch.round(f / step) * step
    y = torch.where(scale[..., None] > 0, b.abs() / scale[..., None], torch.zeros_like(b)).clamp(max=6.0)
    y = torch.where(y < 2, torch.round(y * 2) / 2, torch.where(y < 4, torch.round(y), torch.round(y / 2) * 2))
    code = (y * 2).long()
    code = torch.where(code < 5, code, torch.where(code < 7, 5, torch.where(code < 9, 6, 7))) + 8 * (b < 0)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (scale.half().view(torch.int16) >> 7).to(torch.uint8)


def _store(st, at, k, v, h):
    """Rows k, v [rows, d] of KV heads h to the pool's rows `at`."""
    pages, pool = st["case"]["pages"], st["pool"]
    if pages == "fp4":
        pool[0][at], pool[2][at] = _quant4(k)
        pool[1][at], pool[3][at] = _quant4(v)
    elif pages == "fp8":
        for i, x in enumerate((k, v)):
            code = (x.float() * (1.0 / st["scales"][i][h])).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            pool[i].view(torch.uint8)[at] = code.view(torch.uint8)
    else:
        pool[0][at], pool[1][at] = k.to(torch.bfloat16), v.to(torch.bfloat16)


def _load(st, i, at, h):
    """The values of pool i (0: keys, 1: values) at rows `at` of KV heads h (of at's shape, or one it spreads to), in 32 bits."""
    pages, pool = st["case"]["pages"], st["pool"]
    if pages == "fp4":
        lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
        c = pool[i][at]
        x = lut[torch.stack([c & 15, c >> 4], -1).flatten(-2).long()]
        scale = (pool[2 + i][at].to(torch.int16) << 7).view(torch.float16).float()
        return (x.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2)
    if pages == "fp8":
        x = pool[i].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
        return x * st["scales"][i][h]
    return pool[i][at].float()


def _step(x):
    """The least 2^e, -50 <= e <= 50, with max |x| <= 127 2^e over the last dimension."""
    m, e = torch.frexp(x.abs().amax(-1))
    return torch.exp2((e - 7 + (m > 127.0 / 128.0)).clamp(-50, 50).float())


def _bound(st):
    """Bounds of every full page of the GLOBAL heads, from the pool."""
    case, P = st["case"], st["case"]["page"]
    codes, steps = st["bounds"]
    for a in range(0, len(st["full"]), 1 << 14):                # a few hundred MB of keys at a time
        page, h = st["full"][a:a + (1 << 14)], st["full_head"][a:a + (1 << 14)]
        k = _load(st, 0, page[:, None] * P + torch.arange(P, device=DEV), h[:, None])
        hi, lo = k.amax(1), k.amin(1)
        s = _step(torch.cat([hi, lo], -1))
        codes[0, page] = torch.ceil(hi / s[:, None]).clamp(-127, 127)
        codes[1, page] = torch.floor(lo / s[:, None]).clamp(-127, 127)
        steps[page] = s


def _rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _angles(st):
    p = st["axis_pos"][torch.tensor(st["axis_of"], device=DEV)].T.double()       # [rows, d / 2]
    ang = p[:, None] * st["freq"]
    return torch.cos(ang).float(), torch.sin(ang).float()


def _write(st):
    cos, sin = _angles(st)
    q = _rotate(st["q"].float(), cos, sin).to(torch.bfloat16)
    t, h = st["src"]
    _store(st, st["dst"], _rotate(st["k"].float(), cos, sin)[t, h], st["v"][t, h], h)
    return q, st["pool"][0], st["pool"][1]


def _softmax(s, seen, v, cap):
    """softmax(s) v over the keys that are seen, and the logarithm of its sum."""
    if cap:
        s = cap * torch.tanh(s / cap)
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m.clamp(min=-1e30))
    z = e.sum(-1, keepdim=True)
    return (e @ v) / z, (m + torch.log(z)).squeeze(-1)


def _choose(st, q):
    """Pages kept of each GLOBAL unit [B, G, kept], ascending; a page past the last one where there are fewer."""
    case, P, G = st["case"], st["case"]["page"], st["case"]["globals"]
    j = torch.arange(st["pages"], device=DEV)
    nb = ((st["held"] + P - 1) // P)[:, None, None]
    t = _step(q)
    x = torch.round(q / t[..., None])
    at = (st["page0"][:, :G, None] + j).clamp(max=st["bounds"][1].shape[0] - 1)
    hi, lo = st["bounds"][0][0][at], st["bounds"][0][1][at]
    # whole numbers below 2^21: exact in whatever order they are summed
    score = x.clamp(min=0) @ hi.transpose(-1, -2) + x.clamp(max=0) @ lo.transpose(-1, -2)
    score = (score * t[..., None] * st["bounds"][1][at][:, :, None]).amax(2)
    score = score.masked_fill((j < case["first"]) | (j >= nb - case["newest"]), math.inf).masked_fill(j >= nb, -math.inf)
    some = case["first"] + case["newest"] + case["top"]
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :some]
    order = torch.where(order < nb, order, st["pages"])
    return torch.sort(order, -1)[0]


def _decode(st):
    case, P = st["case"], st["case"]["page"]
    B, G, H, g, d = case["seqs"], case["globals"], case["hkv"], case["hq"] // case["hkv"], case["d"]
    q = st["q"].float().view(B, H, g, d)
    kept = _choose(st, q[:, :G])
    pos = (kept[..., None] * P + torch.arange(P, device=DEV)).flatten(2)
    seen = (pos < st["held"][:, None, None]) & (kept < st["pages"]).repeat_interleave(P, 2)
    at = torch.where(seen, st["page0"][:, :G, None] * P + pos, 0)
    heads = torch.arange(H, device=DEV)

    def attend(qh, at, seen, h):
        k, v = _load(st, 0, at, h), _load(st, 1, at, h)
        return _softmax(qh / math.sqrt(d) @ k.transpose(-1, -2), seen, v, case["cap"])

    a = attend(q[:, :G], at, seen[:, :, None], heads[:G, None])
    b = attend(q[:, G:], st["at"], st["seen"][:, None, None], heads[G:, None])
    out, lse = torch.cat([a[0], b[0]], 1), torch.cat([a[1], b[1]], 1)
    pages = torch.full((B, H, case["first"] + case["newest"] + case["top"]), -1, dtype=torch.int32, device=DEV)
    pages[:, :G, :kept.shape[2]] = torch.where(kept < st["pages"], kept, -1).to(torch.int32)
    return out.reshape(B, case["hq"], d).to(torch.bfloat16), lse.reshape(B, case["hq"]), pages


def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        if kind == "rotate":
            from head_aware_paged_gb300 import sp_rope_axes
            return sp_rope_axes(st["q"], st["k"], st["axis_pos"], st["axis_of"], rope_theta=case["theta"])
        c = st["cache"]
        if kind == "write":
            q = c.append_kv_rope_axes(0, st["ids"], st["cu"], st["q"], st["k"], st["v"], st["axis_pos"], st["axis_of"],
                                      pos=st["start"], rope_theta=case["theta"])
            return q, c.k_pool().view(-1, case["d"]), c.v_pool().view(-1, case["d"])
        for b, (k, v) in enumerate(st["prompts"]):
            c.build(b, 0, k, v)
        res = c.decode_select(0, st["ids"], st["q"], case["top"], sink_pages=case["first"], recent_pages=case["newest"],
                              score_cap=case["cap"] or None)
        for b in range(len(st["prompts"])):
            c.release(b)
        return res
    if kind == "rotate":
        cos, sin = _angles(st)
        return tuple(_rotate(st[x].float(), cos, sin).to(torch.bfloat16) for x in "qk")
    if kind == "write":
        return _write(st)
    if kind == "prompt":
        for k, v, at, (p, h) in st["prompts"]:
            _store(st, at, k[p, h], v[p, h], h)
        _bound(st)
    return _decode(st)


# ---------------------------------------------------------- the definition in 64 bits

def _stored64(case, x, h, scales):
    """Rows x [n, d] (64 bits) of KV head h as the pages' type holds them."""
    if case["pages"] == "bf16":
        return x
    if case["pages"] == "fp8":
        s = scales[h].double()
        y = (x / s).clamp(-448, 448)
        e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
        q = torch.exp2(e - 3)
        return torch.round(y / q) * q * s
    y = x.reshape(x.shape[0], -1, 16)
    top = y.abs().amax(2, keepdim=True) / 6
    q = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -14))) - 3)
    scale = (torch.round(top / q) * q).clamp(max=10240)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=DEV)
    r = y.abs() / scale.clamp(min=2.0 ** -20)
    lo, hi = torch.bucketize(r, mid), torch.bucketize(r, mid, right=True)
    n = torch.where(lo % 2 == 0, lo, hi)                   # a tie takes the even code
    val = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[n]
    return (torch.sign(y) * val * scale).reshape(x.shape)


def _turned64(case, x, pos):
    """x [n, heads, d] turned as complex numbers; pos [3, n]."""
    m = case["d"] // 2
    w = torch.pow(torch.tensor(case["theta"], dtype=torch.float64), -torch.arange(m, dtype=torch.float64) / m).to(DEV)
    turn = torch.stack([pos[a].double() * w[i] for i, a in enumerate(_axis_of(case))], 1)
    z = torch.complex(x[..., :m].double(), x[..., m:].double())
    z = z * torch.polar(torch.ones_like(turn), torch.remainder(turn, 2 * math.pi))[:, None]
    return torch.cat([z.real, z.imag], -1)


def _grid64(x):
    """2^e for each row of x: 127 2^e holds its largest magnitude, 127 2^(e - 1) does not."""
    e = torch.ceil(torch.log2(x.abs().amax(-1).clamp(min=2.0 ** -60) / 127.0))
    e = torch.where(x.abs().amax(-1) > 127.0 * torch.exp2(e), e + 1, e)          # (log2's own rounding)
    e = torch.where(x.abs().amax(-1) <= 127.0 * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp(-50, 50))


def _kept64(case, q, k):
    """Pages kept for the query heads q [g, d] over the stored keys k [n, d]."""
    P, n = case["page"], k.shape[0]
    nb = -(-n // P)
    first, newest, top = case["first"], case["newest"], case["top"]
    if nb <= first + newest + top:
        return list(range(nb))
    mid = nb - first - newest
    blocks = k[first * P:(first + mid) * P].view(mid, P, -1)
    up, dn = blocks.max(1)[0], blocks.min(1)[0]
    s = _grid64(torch.maximum(up.abs(), dn.abs()))[:, None]
    t = _grid64(q)[:, None]
    x = torch.round(q / t)
    worth = torch.full((mid,), -math.inf, dtype=torch.float64, device=DEV)
    for h in range(q.shape[0]):
        each = torch.maximum(x[h] * torch.ceil(up / s), x[h] * torch.floor(dn / s)).sum(1)
        worth = torch.maximum(worth, each * s[:, 0] * t[h])
    worth = worth.tolist()
    best = sorted(range(mid), key=lambda j: (-worth[j], j))[:top]
    return list(range(first)) + sorted(first + j for j in best) + list(range(nb - newest, nb))


def exact(case, seed):
    qkv, history, scales = _inputs(case, seed)
    hq, hkv, d, P, kind = case["hq"], case["hkv"], case["d"], case["page"], case["kind"]
    g, (hist, new), held = hq // hkv, _lengths(case), _held(case)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if kind in ("rotate", "write"):
        pos = _axis_pos(case, seed)
        qt, kt = _turned64(case, q, pos), _turned64(case, k, pos)
        if kind == "rotate":
            return qt, kt
        first, total = _layout(case)
        pools = [torch.zeros(max(1, total) * P, d, dtype=torch.float64, device=DEV) for _ in range(2)]
        row = 0
        for b, (kb, vb) in enumerate(history()):
            for i, (old, x) in enumerate(((kb, kt), (vb, v))):
                x = torch.cat([old[:hist[b]].double(), x[row:row + new[b]].double()])
                for h in range(hkv):
                    slot, kept = _slots(case, h, torch.arange(held[b], device=DEV), held[b])
                    pools[i][first[b * hkv + h] * P + slot[kept]] = x[kept, h]
            row += new[b]
        return qt, pools[0], pools[1]
    out = torch.zeros(case["seqs"], hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(case["seqs"], hq, dtype=torch.float64, device=DEV)
    pages = torch.full((case["seqs"], hkv, case["first"] + case["newest"] + case["top"]), -1, dtype=torch.int32)
    for b, (kb, vb) in enumerate(history()):
        p = torch.arange(held[b], device=DEV)
        for h in range(hkv):
            qh = q[b, h * g:h * g + g].double()
            kh, vh = _stored64(case, kb[:, h].double(), h, scales[0]), _stored64(case, vb[:, h].double(), h, scales[1])
            if h < case["globals"]:
                kept = _kept64(case, qh, kh)
                pages[b, h, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
                see = torch.zeros(-(-held[b] // P), dtype=torch.bool)
                see[kept] = True
                see = see.repeat_interleave(P)[:held[b]].to(DEV)
            else:
                see = (p < case["sink"]) | (p >= held[b] - case["window"])
            s = qh @ kh[see].T / math.sqrt(d)
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            z = torch.logsumexp(s, 1)
            lse[b, h * g:h * g + g] = z
            out[b, h * g:h * g + g] = torch.exp(s - z[:, None]) @ vh[see]
    return out, lse, pages.to(DEV)
