"""Plain attention in 64 bits over explicit rows, for the tests of the capped
scores and of the 4-bit pages.  Test infrastructure only."""
import math

import torch

G, L, R = 0, 1, 2


def visible(pol, pos, i):
    """Which key positions (int64 tensor) the query at position i sees."""
    kind, sink, window, idx = pol
    see = pos <= i
    if kind == L:
        see &= (pos < sink) | (pos > i - window)
    if kind == R:
        see &= torch.isin(pos, torch.tensor(list(idx), dtype=pos.dtype, device=pos.device))
    return see


def attend(q, k, v, rows, pols, cap=None):
    """q [n, hq, d] at positions rows, k, v [m, hkv, d] (64 bits).  Returns the
    output, the log-sum-exp, and what the tolerances are made of: A = sum p |v|
    and S = sum |v| over seen keys (per element), and B = max over seen keys of
    sum |q k| / sqrt(d)."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    pos = torch.arange(k.shape[0], device=q.device)
    out, A, S = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    B = torch.zeros(n, hq, dtype=torch.float64, device=q.device)
    for h in range(hkv):
        see = torch.stack([visible(pols[h], pos, int(i)) for i in rows])
        for j in range(h * g, h * g + g):
            s = q[:, j] @ k[:, h].T / math.sqrt(d)
            if cap:
                s = cap * torch.tanh(s / cap)
            s = s.masked_fill(~see, -math.inf)
            some = see.any(1)
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - torch.where(some, z, torch.zeros_like(z))[:, None])
            out[:, j], A[:, j], lse[:, j] = p @ v[:, h], p @ v[:, h].abs(), z
            S[:, j] = see.double() @ v[:, h].abs()
            b = (q[:, j].abs() @ k[:, h].abs().T / math.sqrt(d)).masked_fill(~see, 0.0)
            B[:, j] = b.amax(1)
    return out, lse, A, B, S


def check(out, lse, ref, p_eps, score_eps, what="", cap=None):
    """|out - o| <= half a bf16 step of o + (p_eps + 2 ds) A + p_abs S, and |lse - z| <=
    ds + fp32 slack, where ds = score_eps B is how far a score may be off:
    softmax weights then move by e^(2 ds) - 1 at most, and P's own rounding is
    p_eps of each.  p_abs: P in f16 (p_eps 2^-11) is off by up to 2^-25, half
    its least step, where it is small, next to a largest weight of 1 or more
    (a key that is e^-19 of the largest weighs 2^-27: the product drops it).  fp32 slack: 256 terms of 2^-24 for sums, 2^-20 (1 + |z|)
    for exp2 / log2; the cap's tanh adds cap * 3e-7."""
    o, z, A, B, S = ref
    p_abs = 2.0 ** -25 if p_eps == 2.0 ** -11 else 0.0
    ds = score_eps * B + 2.0 ** -16 * B + 2.0 ** -20 + (3e-7 * cap if cap else 0.0)
    got = out.double()
    assert torch.isfinite(got).all(), what
    tol = 2.0 ** -8 * o.abs() + (p_eps + 2.0 ** -15 + torch.expm1(2 * ds)[..., None]) * A + p_abs * S + 1e-30
    worst = ((got - o).abs() / tol).max().item()
    assert worst <= 1.0, "%s: out %.3g of its tolerance" % (what, worst)
    if lse is not None:
        none = torch.isneginf(z)
        assert torch.equal(torch.isneginf(lse), none), what
        tol = ds + 2.0 ** -19 * (1 + z.abs().nan_to_num(0, 0, 0))
        worst = ((lse.double() - z).abs()[~none] / tol[~none]).max().item() if (~none).any() else 0.0
        assert worst <= 1.0, "%s: lse %.3g of its tolerance" % (what, worst)
