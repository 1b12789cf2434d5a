"""4-bit K/V pages -- quantisation, dequantisation and byte layout, plain
definitions in float64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

A row's 16 neighbouring dimensions share a scale: an unsigned float of 5
exponent and 3 mantissa bits (0, the subnormals m * 2^-17, and
(1 + m/8) * 2^(e - 15)), at most 10240, nearest to amax / 6 with ties to the
even code.  An element is the e2m1 value (0, .5, 1, 1.5, 2, 3, 4, 6 and their
negatives) nearest to x / scale, ties to the even code, at most 6.  Channel
scales divide first, as fp32(x * fp32(1 / s)).
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([(c & 7) * 2.0 ** -17 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 15)
                   for c in range(227)])            # SCALES[226] = 10240


def _nearest(x: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Index of the nearest of the ascending values (ties to the even index)."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    below, above = x - values[lo], values[hi] - x
    take = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(take, hi, lo)


def quantize(x, channel=None):
    """Codes (0..15) and scale codes of rows x [..., d]; channel [d] fp32."""
    x = np.asarray(x, dtype=np.float64)
    if channel is not None:
        inv = (np.float32(1.0) / np.asarray(channel, np.float32)).astype(np.float32)
        x = (x.astype(np.float32) * inv).astype(np.float64)
    b = x.reshape(*x.shape[:-1], -1, 16)
    sc = _nearest(np.minimum(np.abs(b).max(axis=-1) / 6.0, SCALES[-1]), SCALES)
    s = SCALES[sc][..., None]
    y = np.divide(np.abs(b), s, out=np.zeros_like(b), where=s > 0)
    code = _nearest(np.minimum(y, 6.0), E2M1) + 8 * ((b < 0) & (s > 0))
    return code.reshape(x.shape).astype(np.uint8), sc.astype(np.uint8)


def dequantize(code, sc, channel=None):
    code = np.asarray(code)
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    out = (v.reshape(*v.shape[:-1], -1, 16) * SCALES[np.asarray(sc)][..., None]).reshape(v.shape)
    return out if channel is None else out * np.asarray(channel, np.float32).astype(np.float64)


def stored(x, channel=None):
    """The value that rows x are held as."""
    return dequantize(*quantize(x, channel), channel)


# Places inside a group of 16 slots (1152 bytes: 1024 of codes, 128 of scales),
# written out as the two fragments read them: lane (g, j) of a K fragment reads
# 16 bytes at row position g (and g + 8), lane (g, j) of a V fragment 8 bytes of
# slots j, j + 4, j + 8, j + 12.
def k_row(slot: int) -> int:
    order = [0, 4, 1, 5, 2, 6, 3, 7, 8, 12, 9, 13, 10, 14, 11, 15]   # slot at each position
    return order.index(slot)


def read_row(group: np.ndarray, slot: int, value: bool):
    """Codes [128] and scale codes [8] of one slot of a group (uint8 [1152])."""
    code, sc = np.zeros(128, np.uint8), np.zeros(8, np.uint8)
    for b in range(8):
        if value:
            at = slot * 64 + (b ^ (4 if slot % 4 >= 2 else 0)) * 8
            sc[b] = group[1024 + 16 * b + 4 * (slot % 4) + slot // 4]
        else:
            r = k_row(slot)
            at = r * 64 + b * 8
            sc[b] = group[1024 + 16 * (r % 8) + 4 * (b // 2) + 2 * (r // 8) + b % 2]
        byte = group[at:at + 8]
        code[16 * b:16 * b + 16:2], code[16 * b + 1:16 * b + 16:2] = byte & 15, byte >> 4
    return code, sc
