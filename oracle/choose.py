"""The choice of pages for a decode query -- the plain definition.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Bounds of a page's keys in every dimension, on a grid of a power of two; the
score of a page for a query head; the pages that are kept.  All in integers and
float64 powers of two, so every value is exact.
"""
from __future__ import annotations

import numpy as np


def grid(x) -> np.ndarray:
    """The least 2^e, -50 <= e <= 50, with max |x| <= 127 * 2^e over the last axis."""
    # (fp32 values next to 127 * 2^e stay on their side of 2^e in the float64 quotient)
    m, e = np.frexp(np.max(np.abs(np.asarray(x, np.float64)), axis=-1) / 127.0)
    e = np.where(np.isinf(m), 50, np.where(m == 0.5, e - 1, np.where(m == 0.0, -50, e)))
    return np.ldexp(1.0, np.clip(e, -50, 50))


def bounds(keys):
    """keys [n, d] of one page: (upper codes, lower codes, step)."""
    k = np.asarray(keys, np.float64)
    hi, lo = k.max(0), k.min(0)
    s = grid(np.concatenate([hi, lo]))
    return (np.clip(np.ceil(hi / s), -127, 127).astype(np.int64),
            np.clip(np.floor(lo / s), -127, 127).astype(np.int64), float(s))


def query(q):
    """One query head q [d]: (codes, step).  np.rint rounds ties to even."""
    t = grid(q)
    return np.clip(np.rint(np.asarray(q, np.float64) / t), -127, 127).astype(np.int64), float(t)


def scores(qs, pages):
    """Of every page's bounds for the query heads qs [g, d] of their KV head."""
    codes = [query(q) for q in qs]
    return [max(float(np.maximum(x * hi, x * lo).sum()) * s * t for x, t in codes) for hi, lo, s in pages]


def score(qs, page) -> float:
    return scores(qs, [page])[0]


def kept(scores, nb: int, first: int, newest: int, top: int):
    """Pages kept of nb, ascending; scores[j] of page j (read for candidates only)."""
    if nb <= first + newest + top:
        return list(range(nb))
    cand = range(first, nb - newest)
    best = sorted(cand, key=lambda j: (-scores[j], j))[:top]
    return list(range(first)) + sorted(best) + list(range(nb - newest, nb))
