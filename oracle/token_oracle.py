"""CPU oracle of the 4-bit products with scales per group and of the sampler.

TEST INFRASTRUCTURE ONLY, like q2_oracle: NumPy float64 and plain loops, written
from the definitions; it shares no code with the library.

* weight: (code - zero) * scale, codes two per byte, low nibble = even input; one
  scale and zero point per group of inputs, the zero point 8, an f16 or a 4-bit code
  (two per byte, low nibble = even group).
* sample: tokens in descending order of their logits, equal ones by lower token,
  masked ones (-inf, NaN) left out; p = exp((logit - best) / temperature); min-p,
  top-k and top-p leave a beginning of that order each; the first token whose
  cumulative p exceeds u times the sum of what is left.
"""
from __future__ import annotations

import math

import numpy as np


def nibbles(packed: np.ndarray, count: int) -> np.ndarray:
    """The first `count` 4-bit codes of each row of bytes."""
    out = np.zeros((packed.shape[0], 2 * packed.shape[1]), np.int64)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out[:, :count]


def weight(packed: np.ndarray, scale: np.ndarray, zero) -> np.ndarray:
    """float64 weight [N, K] of codes u8 [N, K/2], float scales [N, G] and zero points (None, u8 codes or floats)."""
    n, k = packed.shape[0], 2 * packed.shape[1]
    groups = scale.shape[1]
    if zero is None:
        z = np.full((n, groups), 8.0)
    elif zero.dtype == np.uint8:
        z = nibbles(zero, groups).astype(np.float64)
    else:
        z = zero.astype(np.float64)
    w = np.zeros((n, k))
    codes = nibbles(packed, k)
    for i in range(k):
        g = i // (k // groups)
        w[:, i] = (codes[:, i] - z[:, g]) * scale[:, g].astype(np.float64)
    return w


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability) of one row."""
    logits = np.asarray(logits, np.float64)
    order = [int(i) for i in np.lexsort((np.arange(len(logits)), -logits)) if logits[i] > -math.inf]   # NaN: false
    if not order:
        return -1, 0.0
    if not temperature > 0 or top_k == 1 or top_p <= 0 or min_p > 1:
        return order[0], 1.0
    l = logits[order]
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.exp((l - l[0]) / temperature)
    p[np.isnan(p)] = 0.0
    p[l == l[0]] = 1.0
    n = len(p)
    if min_p > 0:
        n = int(np.sum(p >= min_p))                        # p falls along the order
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        c = np.cumsum(p[:n])
        n = int(np.argmax(c >= top_p * c[-1])) + 1
    c = np.cumsum(p[:n])
    u = u if u > 0 else 0.0                                # NaN too
    above = np.nonzero(c > u * c[-1])[0]
    at = int(above[0]) if len(above) and u < 1 else int(np.nonzero(p[:n])[0][-1])
    return order[at], p[at] / c[-1]


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token i32 [B], probability float64 [B]); each setting a number or one per row."""
    def of(s, i):
        return s if np.ndim(s) == 0 else s[i]

    out = [sample_row(logits[i], float(u[i]), float(of(temperature, i)), int(of(top_k, i)), float(of(top_p, i)),
                      float(of(min_p, i))) for i in range(len(logits))]
    return np.array([t for t, _ in out], np.int32), np.array([p for _, p in out], np.float64)
