"""Oracle of the AdamW step and of its 8-bit states.

TEST INFRASTRUCTURE ONLY.  Only tests/, __graft_entry__.smoke() and the
cpu_baseline leg of bench.py may import this module; the product path never
imports, calls or links it.

Source: AdamW (Loshchilov and Hutter, "Decoupled Weight Decay
Regularization", 2019, Algorithm 2), in float64:
    m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
    p = p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
8-bit states: runs of 256 elements, each value x stored as the e4m3 code
nearest to x / scale, scale = largest |x| / 448.  e4m3 (OCP 8-bit floating
point, 1 sign, 4 exponent, 3 mantissa bits, bias 7) holds 2^-9 i below 2^-6
and (1 + i / 8) 2^e above, up to 448; 0x7F is NaN.

encode_random takes the code above x / scale instead of the one below where a
uniform number u is below (x - lo) / (hi - lo), or of the squares for roots, so
that the expected value (square) is x (x^2).
"""

from __future__ import annotations

import numpy as np

BLOCK = 256


def step(p, g, m, v, t, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0):
    """(p, m, v) after step t (from 1)."""
    p, g, m, v = (np.asarray(x, dtype=np.float64) for x in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** t), v / (1 - beta2 ** t)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v


def code_values() -> np.ndarray:
    """The 256 codes' values (NaN at 0x7F and 0xFF)."""
    out = np.empty(256)
    for c in range(256):
        e, i = (c >> 3) & 15, c & 7
        x = i * 2.0 ** -9 if e == 0 else (1 + i / 8) * 2.0 ** (e - 7)
        out[c] = (-x if c & 128 else x) if (c & 127) != 127 else np.nan
    return out


def decode(codes, scales):
    """The values of codes [n] with one scale per run."""
    codes = np.asarray(codes, dtype=np.uint8)
    return code_values()[codes] * np.repeat(np.asarray(scales, dtype=np.float64), BLOCK)[: codes.size]


def encode(x, root: bool = False):
    """(codes, scales) of x [n]; root: the values are square roots of v,
    and one above zero takes at least the smallest code."""
    x = np.asarray(x, dtype=np.float64)
    table = code_values()[:127]
    codes, scales = np.zeros(x.size, dtype=np.uint8), []
    for a in range(0, x.size, BLOCK):
        part = x[a:a + BLOCK]
        top = np.abs(part).max()
        scales.append(top / 448 if top >= 2.0 ** -100 else 0.0)
        if scales[-1] == 0.0:
            continue
        for i, val in enumerate(part):
            mag = abs(val) / scales[-1]
            d = np.abs(table - mag)
            near = np.flatnonzero(d == d.min())
            c = int(near[0]) if near.size == 1 or near[0] % 2 == 0 else int(near[1])
            if root and val > 0:
                c = max(c, 1)
            codes[a + i] = c | (128 if val < 0 else 0)
    return codes, np.array(scales)


def encode_random(x, u, root: bool = False):
    """(codes, scales) of x [n] with uniform numbers u [n] in [0, 1)."""
    x, u = np.asarray(x, dtype=np.float64), np.asarray(u, dtype=np.float64)
    table = code_values()[:127]
    starts = np.arange(0, x.size, BLOCK)
    top = np.maximum.reduceat(np.abs(x), starts)
    scales = np.where(top >= 2.0 ** -100, top / 448, 0.0)
    per = np.repeat(scales, BLOCK)[: x.size]
    mag = np.where(per > 0, np.abs(x) / np.where(per > 0, per, 1.0), 0.0)
    if root:
        mag = np.where(mag > 0, np.maximum(mag, table[1]), mag)
    below = np.clip(np.searchsorted(table, mag, side="right") - 1, 0, 125)
    power = 2 if root else 1
    lo, hi = table[below] ** power, table[below + 1] ** power
    codes = below + (u < (mag ** power - lo) / (hi - lo))
    return np.where(x < 0, codes | 128, codes).astype(np.uint8), scales
