"""Performance cases of the cache's write-with-rotation, 4-bit pages and capped scores.

Three operators, in the calls that serve a model:

  write   `append_kv_rope`: the rotary embedding of new queries and keys, and the
          rotated keys and the values written into their heads' pages
  decode  one query a sequence over the pages (bf16, FP8 or 4-bit), the scores
          capped by cap * tanh(score / cap) or as they are
  chunk   the same for a chunk of new rows over paged history and itself
  step    a serving step: the new token's write, then its decode

`run` computes them with elementary torch operations (own = False) or with the
package (own = True).  Writes go to positions that the sequences hold already, so
that a pass can be repeated.  KV heads 0 .. globals-1 see everything, the others
their `sink` first tokens and the newest `window`.

4-bit pages: 16 neighbouring dimensions share a scale with 5 exponent and 3 mantissa
bits (an f16 with its low 7 bits zero), the value nearest amax / 6 (ties to even, at
most 10240); an element is the e2m1 value (0, .5, 1, 1.5, 2, 3, 4, 6, signed)
nearest x / scale (ties to an even mantissa, at most 6).
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ROW_BYTES = {"bf16": 2.0, "fp8": 1.0, "fp4": 0.5625}     # per element, scales included


def listed():
    """A head layout of 32 query and 8 KV heads with one GLOBAL head of eight, sink 4 and
    windows of 1024 to 2048 is the repository's own; page 64 too."""
    base = dict(hq=32, hkv=8, d=128, page=64, globals=1, sink=4, window=1024, ragged=False)
    return [
        # the new token of each of 64 sequences in a serving step: latency
        dict(base, name="write_step_64", kind="write", pages="bf16", seqs=64, hist=500, new=1, theta=500000.0),
        # a whole prompt written after its projections
        dict(base, name="write_prompt_8k", kind="write", pages="bf16", seqs=1, hist=0, new=8192, theta=500000.0),
        # several short prompts of odd lengths, a small model's heads
        dict(base, name="write_ragged_d64", kind="write", pages="bf16", seqs=7, hist=90, new=333, theta=10000.0,
             hq=14, hkv=2, d=64, page=16, window=100, ragged=True),
        # one user's conversation on 4-bit pages: the smallest step
        dict(base, name="step_fp4_single", kind="step", pages="fp4", cap=0.0, seqs=1, hist=2047, new=1, theta=500000.0),
        # a batch of odd lengths with an odd group of query heads
        dict(base, name="step_fp4_ragged", kind="step", pages="fp4", cap=0.0, seqs=19, hist=9001, new=1,
             theta=10000.0, hq=35, hkv=5, globals=2, window=777, ragged=True),
        # 32 sequences of 32K tokens: the decode batch that the benchmark runs on bf16 pages
        dict(base, name="decode_fp4_32x32k", kind="decode", pages="fp4", cap=0.0, seqs=32, hist=32768, window=2048),
        # capped scores over bf16 pages, every head GLOBAL
        dict(base, name="decode_cap_32x8k", kind="decode", pages="bf16", cap=50.0, seqs=32, hist=8192, globals=8),
        # capped scores over FP8 pages, odd lengths
        dict(base, name="decode_cap_fp8_ragged", kind="decode", pages="fp8", cap=30.0, seqs=9, hist=20001,
             globals=3, window=1500, ragged=True),
        # the last chunk of a long prompt on 4-bit pages
        dict(base, name="chunk_fp4_2k_of_18k", kind="chunk", pages="fp4", cap=0.0, seqs=1, hist=16384, new=2048),
        # short chunks of several sequences on 4-bit pages, capped
        dict(base, name="chunk_fp4_cap_ragged", kind="chunk", pages="fp4", cap=30.0, seqs=5, hist=3001, new=211,
             globals=3, ragged=True),
        # an 8K prompt's layer with capped scores
        dict(base, name="chunk_cap_8k", kind="chunk", pages="bf16", cap=50.0, seqs=1, hist=0, new=8192),
        # short chunks with one query head a KV head, head_dim 64, small pages
        dict(base, name="chunk_cap_ragged_d64", kind="chunk", pages="bf16", cap=30.0, seqs=6, hist=700, new=150,
             hq=12, hkv=12, d=64, page=16, globals=5, window=300, ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["write", "step", "decode", "decode", "chunk", "chunk"])
    pages = rng.choice(["bf16", "fp8", "fp4", "fp4"]) if kind != "write" else "bf16"
    d = 128 if pages != "bf16" else rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8])
    c = dict(kind=kind, pages=pages, d=d, hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 4, 7, 8, 12]),
             page=rng.choice([16, 32, 64, 64, 128]), globals=rng.randint(0, hkv), sink=rng.choice([0, 4, 4, 37]),
             window=_log(rng, 1, 4096), ragged=rng.random() < 0.6, theta=rng.choice([10000.0, 500000.0]))
    if kind == "write":
        c["seqs"], c["hist"], c["new"] = (_log(rng, 1, 128), _log(rng, 1, 600), 1) if rng.random() < 0.5 else \
            (rng.randint(1, 4), _log(rng, 1, 300), _log(rng, 2, 2048))
        return c
    c["cap"] = rng.choice([0.0, 20.0, 50.0]) if pages == "fp4" else rng.choice([1.5, 20.0, 30.0, 50.0])
    if kind == "chunk":
        c["seqs"], c["hist"], c["new"] = rng.randint(1, 4), _log(rng, 1, 8192), _log(rng, 1, 2048)
        while c["seqs"] * c["hq"] * c["new"] * (c["hist"] + c["new"]) > 1 << 31:
            c["hist"], c["new"] = 1 + c["hist"] // 2, 1 + c["new"] // 2
    else:
        c["seqs"], c["hist"], c["new"] = _log(rng, 1, 32), _log(rng, 1, 32767), 1
    return c


# ----------------------------------------------------------- shapes and layout

def _lengths(case):
    """Tokens held before the new ones, and new tokens, of each sequence."""
    r = random.Random("%(seqs)d %(hist)d" % case)
    f = [1.0 if not case["ragged"] else math.exp(r.uniform(-1.5, 0.0)) for _ in range(case["seqs"])]
    new = case.get("new", 0) if case["kind"] != "decode" else 0
    return [max(int(case["kind"] == "decode"), int(case["hist"] * x)) for x in f], [max(1, int(new * x)) if new else 0 for x in reversed(f)]


def _unit(case, h, n):
    """(pages, LOCAL?, sink pages, ring slots) of KV head h that holds n tokens."""
    P = case["page"]
    if h < case["globals"]:
        return -(-n // P), False, 0, 0
    ring = -(-case["window"] // P) + 1
    s = case["sink"]
    return -(-min(n, s) // P) + min(ring, -(-max(0, n - s) // P)), True, -(-s // P), ring * P


def _held(case):
    """Tokens in the pages when `run` is called: a write's are rewritten, a chunk's are not there yet."""
    h, n = _lengths(case)
    return h if case["kind"] in ("chunk", "decode") else [a + b for a, b in zip(h, n)]


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


def _seen(case, h, n):
    """Keys that a query at position n - 1 sees."""
    return n if h < case["globals"] else min(n, case["sink"] + case["window"])


def work(case):
    hist, new = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g, row = hq // hkv, 2 * d * ROW_BYTES[case["pages"]]
    byt = flo = 0.0
    for a, c, n in zip(hist, new, _held(case)):
        for h in range(hkv):
            _, local, _, ring = _unit(case, h, n)
            kept = c if not local else sum(1 for p in range(a, n) if p < case["sink"] or p >= n - ring)
            if case["kind"] in ("write", "step"):
                byt += kept * (4 * d + row) + c * g * 4 * d
                flo += 3 * d * (kept + c * g)
            if case["kind"] in ("decode", "step"):
                byt += _seen(case, h, n) * row + g * (4 * d + 4)
                flo += 4 * d * g * _seen(case, h, n)
            if case["kind"] == "chunk":
                lo = 0 if not local else max(0, a + 1 - case["window"])
                byt += (min(a, lo and case["sink"]) + a - min(a, max(lo, lo and case["sink"]))) * row
                byt += c * (4 * d + g * (4 * d + 4))
                flo += 4 * d * g * sum(_seen(case, h, i + 1) for i in range(a, a + c))
    return {"bytes": byt, "flops": flo}


# -------------------------------------------------------------------- inputs

def _inputs(case, seed):
    """The new tokens' projections as one packed tensor, as a fused projection leaves
    them, and a generator of each sequence's history.  Keys have a few strong channels."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    hist, new = _lengths(case)
    rows = sum(new) if case["kind"] != "decode" else case["seqs"]
    strong = torch.ones(hkv, d, device=DEV)
    strong[:, torch.randperm(d, generator=g, device=DEV)[:4]] = 6.0
    qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g, device=DEV)
    qkv[:, :hq] *= 2.0 if case.get("cap") else 1.0
    qkv[:, hq:hq + hkv] *= 0.5 * strong
    qkv = qkv.to(torch.bfloat16)

    def history():
        for n in _held(case):
            k = (torch.randn(n, hkv, d, generator=g, device=DEV) * (0.5 * strong)).to(torch.bfloat16)
            yield k, torch.randn(n, hkv, d, generator=g, device=DEV).to(torch.bfloat16)

    # FP8 channel scales: powers of two, as a calibration rounds them
    ex = torch.randint(-6, -2, (2, hkv, d), generator=g, device=DEV).float()
    return qkv, history, torch.exp2(ex)


def prepare(case, seed):
    qkv, history, scales = _inputs(case, seed)
    hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["page"]
    hist, new = _lengths(case)
    cu = [0]
    for c in (new if case["kind"] != "decode" else [1] * case["seqs"]):
        cu.append(cu[-1] + c)
    half = torch.arange(d // 2, dtype=torch.float64)
    st = dict(case=case, cu=cu, start=list(hist), ids=list(range(case["seqs"])),
              q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
    if case["kind"] == "chunk":
        st.update(q=st["q"].contiguous(), k=st["k"].contiguous(), v=st["v"].contiguous())
    if case["kind"] == "decode":
        st.update(q=st["q"].contiguous())
    first, total = _layout(case)
    held = _held(case)
    if own:
        from head_aware_paged_gb300 import GLOBAL, KV_BF16, KV_FP4, KV_FP8, LOCAL, Config, Policy, SegPagedCache
        cache = SegPagedCache(Config(
            num_layers=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P, max_seqs=case["seqs"],
            max_seq_len=max([a + b for a, b in zip(hist, new)] + [case["window"], case["sink"]]) + 1, num_pages=max(1, total),
            max_tokens=max(max(held), cu[-1]), max_batch=case["seqs"],
            kv_dtype={"bf16": KV_BF16, "fp8": KV_FP8, "fp4": KV_FP4}[case["pages"]]))
        if case["pages"] == "fp8":
            cache.set_kv_scales(0, scales[0].cpu().numpy(), scales[1].cpu().numpy())
        row = [Policy(GLOBAL) if h < case["globals"] else Policy(LOCAL, case["sink"], case["window"]) for h in range(hkv)]
        for b, (k, v) in enumerate(history()):
            cache.set_policy(b, [row])
            if held[b]:
                cache.build(b, 0, k, v)
        st["cache"] = cache
        return st
    # the plain form's pools, in the same page order
    rows = max(1, total) * P
    if case["pages"] == "fp4":
        pool = [torch.zeros(rows, d // 2, dtype=torch.uint8, device=DEV) for _ in range(2)]
        pool += [torch.zeros(rows, d // 16, dtype=torch.uint8, device=DEV) for _ in range(2)]
    else:
        t = torch.bfloat16 if case["pages"] == "bf16" else torch.float8_e4m3fn
        pool = [torch.zeros(rows, d, device=DEV).to(t) for _ in range(2)]
    st.update(pool=pool, scales=scales, freq=(case.get("theta", 1e4) ** (-2.0 * half / d)).to(DEV))
    dst, src = [], []
    span = max([1] + held)
    where = torch.zeros(case["seqs"], hkv, span, dtype=torch.int64, device=DEV)
    for b, (k, v) in enumerate(history()):
        p = torch.arange(held[b], device=DEV)
        for h in range(hkv):
            slot, kept = _slots(case, h, p, held[b])
            at = first[b * hkv + h] * P + slot
            _store(st, at[kept], k[kept, h], v[kept, h], torch.tensor(h, device=DEV))
            where[b, h, :held[b]] = torch.where(kept, at, 0)
            if case["kind"] in ("write", "step"):
                w = torch.arange(hist[b], held[b], device=DEV)
                w = w[kept[hist[b]:]]
                dst.append(at[w])
                src.append(torch.stack([cu[b] + w - hist[b], torch.full_like(w, h)]))
    if dst:
        st["dst"], st["src"] = torch.cat(dst), torch.cat(src, 1)
        st["pos"] = torch.cat([torch.arange(a, a + c, device=DEV) for a, c in zip(hist, new)])
    n = torch.tensor(held, device=DEV)
    if case["kind"] == "chunk":
        c = torch.tensor(new, device=DEV)
        r = torch.arange(max(new), device=DEV)
        st["take"] = torch.tensor(cu[:-1], device=DEV)[:, None] + r.clamp(max=int(c.max()) - 1).minimum(c[:, None] - 1)
        st["back"] = torch.cat([b * max(new) + torch.arange(x, device=DEV) for b, x in enumerate(new)])
        st["qpos"] = n[:, None] + r
        kp = torch.arange(span, device=DEV)
        far = torch.tensor(1 << 40, device=DEV)
        st["kpos"] = torch.cat([torch.where(kp < n[:, None], kp, far), torch.where(r < c[:, None], n[:, None] + r, far)], 1)
        st["where"] = where
    elif case["kind"] != "write":
        # the keys that each unit's query sees, padded to the longest of the head class
        s, w = case["sink"], case["window"]
        gl = torch.arange(span, device=DEV).expand(case["seqs"], span)
        lo = (n[:, None] - w).clamp(min=s)
        lp = torch.cat([torch.arange(s, device=DEV).expand(case["seqs"], s), lo + torch.arange(w, device=DEV)], 1)[:, :max(1, min(s + w, span + s))]
        st["seen"] = [gl < n[:, None], lp < n[:, None]]
        G = case["globals"]
        pick = lambda rows, at: torch.gather(rows, 2, at[:, None].clamp(max=span - 1).expand(-1, rows.shape[1], -1))  # noqa: E731
        st["at"] = [pick(where[:, :G], gl), pick(where[:, G:], lp)]
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


def _load(st, i, at, h0):
    """The values of pool i (0: keys, 1: values) at rows [B, H, S], KV heads from h0, in 32 bits."""
    pages, pool = st["case"]["pages"], st["pool"]
    if pages == "fp4":
        lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
        c = pool[i][at]
        x = lut[torch.stack([c & 15, c >> 4], -1).flatten(-2).long()]
        scale = (pool[2 + i][at].to(torch.int16) << 7).view(torch.float16).float()
        return (x.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2)
    if pages == "fp8":
        x = pool[i].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
        return x * st["scales"][i][h0:h0 + at.shape[1], None]
    return pool[i][at].float()


def _rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _write(st):
    """Rotated queries; rotated keys and the values go to the pool."""
    wide = torch.float64 if st["case"]["pages"] == "fp4" else torch.float32
    ang = st["pos"].double()[:, None, None] * st["freq"]
    cos, sin = torch.cos(ang).to(wide), torch.sin(ang).to(wide)
    q = _rotate(st["q"].float(), cos.float(), sin.float()).to(torch.bfloat16)
    t, h = st["src"]
    _store(st, st["dst"], _rotate(st["k"].to(wide), cos, sin)[t, h], st["v"][t, h], h)
    return q


def _softmax(s, seen, v, cap):
    """softmax(s) v over the keys that are seen, and the logarithm of its sum."""
    if cap:
        s = cap * torch.tanh(s / cap)
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m.clamp(min=-1e30))
    z = e.sum(-1, keepdim=True)
    return (e @ v) / z, (m + torch.log(z)).squeeze(-1)


def _decode(st, q):
    case = st["case"]
    B, G, g, d = case["seqs"], case["globals"], case["hq"] // case["hkv"], case["d"]
    q = q.float().view(B, case["hkv"], g, d) / math.sqrt(d)

    def heads(qh, c, h0):
        k, v = _load(st, 0, st["at"][c], h0), _load(st, 1, st["at"][c], h0)
        return _softmax(qh @ k.transpose(-1, -2), st["seen"][c][:, None, None], v, case["cap"])

    a, b = heads(q[:, :G], 0, 0), heads(q[:, G:], 1, G)
    out, lse = torch.cat([a[0], b[0]], 1), torch.cat([a[1], b[1]], 1)
    return out.reshape(B, case["hq"], d).to(torch.bfloat16), lse.reshape(B, case["hq"])


def _chunk(st):
    case = st["case"]
    G, g, d = case["globals"], case["hq"] // case["hkv"], case["d"]
    q = st["q"][st["take"]].float().unflatten(2, (case["hkv"], g)).permute(0, 2, 3, 1, 4) / math.sqrt(d)
    join = lambda i, x: torch.cat([_load(st, i, st["where"], 0), x[st["take"]].float().transpose(1, 2)], 2)  # noqa: E731
    k, v = join(0, st["k"])[:, :, None], join(1, st["v"])[:, :, None]
    i, p = st["qpos"][:, None, None, :, None], st["kpos"][:, None, None, None]
    near = (p < case["sink"]) | (p > i - case["window"])
    a = _softmax(q[:, :G] @ k[:, :G].transpose(-1, -2), p <= i, v[:, :G], case["cap"])
    b = _softmax(q[:, G:] @ k[:, G:].transpose(-1, -2), (p <= i) & near, v[:, G:], case["cap"])
    out = torch.cat([a[0], b[0]], 1).permute(0, 3, 1, 2, 4).reshape(-1, case["hq"], d)
    lse = torch.cat([a[1], b[1]], 1).permute(0, 3, 1, 2).reshape(-1, case["hq"])
    return out[st["back"]].to(torch.bfloat16), lse[st["back"]].contiguous()


def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        c, cap = st["cache"], case.get("cap") or None
        if kind == "chunk":
            return c.prefill(0, st["ids"], st["cu"], st["q"], st["k"], st["v"], score_cap=cap)
        if kind == "decode":
            return c.decode(0, st["ids"], st["q"], score_cap=cap)
        q = c.append_kv_rope(0, st["ids"], st["cu"], st["q"], st["k"], st["v"], pos=st["start"], rope_theta=case["theta"])
        return (q, c.k_pool().view(-1, case["d"]), c.v_pool().view(-1, case["d"])) if kind == "write" else \
            (q, *c.decode(0, st["ids"], q, score_cap=cap))
    if kind == "chunk":
        return _chunk(st)
    if kind == "decode":
        return _decode(st, st["q"])
    q = _write(st)
    return (q, st["pool"][0], st["pool"][1]) if kind == "write" else (q, *_decode(st, q))


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
    """x [n, heads, d] turned as complex numbers by its positions' angles."""
    m = case["d"] // 2
    w = torch.pow(torch.tensor(case["theta"], dtype=torch.float64), -torch.arange(m, dtype=torch.float64) / m).to(DEV)
    ang = torch.remainder(pos.double()[:, None] * w, 2 * math.pi)
    z = torch.complex(x[..., :m].double(), x[..., m:].double()) * torch.polar(torch.ones_like(ang), ang)[:, None]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    qkv, history, scales = _inputs(case, seed)
    hq, hkv, d, P, kind = case["hq"], case["hkv"], case["d"], case["page"], case["kind"]
    g, (hist, new), held = hq // hkv, _lengths(case), _held(case)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    outs, lses, turned = [], [], []
    first, total = _layout(case)
    pools = [torch.zeros(max(1, total) * P, d, dtype=torch.float64, device=DEV) for _ in range(2)] if kind == "write" else None
    row = 0
    for b, (kb, vb) in enumerate(history()):
        c = new[b] if kind != "decode" else 1
        qb, kn, vn = q[row:row + c].double(), k[row:row + c].double(), v[row:row + c].double()
        row += c
        kb, vb = kb.double(), vb.double()
        if kind in ("write", "step"):
            pos = torch.arange(hist[b], held[b], device=DEV)
            qb = _turned64(case, qb, pos)
            kb = torch.cat([kb[:hist[b]], _turned64(case, kn, pos)])
            vb = torch.cat([vb[:hist[b]], vn])
            turned.append(qb)
            if kind == "step":
                qb = qb.to(torch.bfloat16).double()        # the step's decode reads them in this type
        keys = torch.arange(held[b] + (c if kind == "chunk" else 0), device=DEV)
        at = torch.arange(hist[b], hist[b] + c, device=DEV) if kind == "chunk" else torch.tensor([held[b] - 1], device=DEV)
        o = torch.zeros(c, hq, d, dtype=torch.float64, device=DEV)
        z = torch.zeros(c, hq, dtype=torch.float64, device=DEV)
        for h in range(hkv):
            if kind == "write":
                slot, kept = _slots(case, h, keys, held[b])
                for i, x in enumerate((kb, vb)):
                    pools[i][first[b * hkv + h] * P + slot[kept]] = x[kept, h]
                continue
            kh, vh = _stored64(case, kb[:, h], h, scales[0]), _stored64(case, vb[:, h], h, scales[1])
            if kind == "chunk":
                kh, vh = torch.cat([kh, kn[:, h]]), torch.cat([vh, vn[:, h]])
            see = keys[None] <= at[:, None]
            if h >= case["globals"]:
                see &= (keys[None] < case["sink"]) | (keys[None] > at[:, None] - case["window"])
            for j in range(h * g, h * g + g):
                s = qb[:, j] @ kh.T / math.sqrt(d)
                if case["cap"]:
                    s = case["cap"] * torch.tanh(s / case["cap"])
                s = torch.where(see, s, torch.full_like(s, -math.inf))
                z[:, j] = torch.logsumexp(s, 1)
                o[:, j] = torch.exp(s - z[:, j, None]) @ vh
        outs.append(o)
        lses.append(z)
    if kind == "write":
        return torch.cat(turned), pools[0], pools[1]
    tail = (torch.cat(outs), torch.cat(lses))
    return tail if kind != "step" else (torch.cat(turned), *tail)
