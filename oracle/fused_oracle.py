"""CPU oracle of the fused and grouped linears, the router and the combination.

TEST INFRASTRUCTURE ONLY, like q2_oracle: NumPy float64 and plain loops, written
from the definitions; it shares no code with the library.

* fused: y = residual + gate * a with a = act(z + bias), or, for a gated weight
  of 2 n rows, act(z + bias)[:n] * (z + bias)[n:]; z = x W^T (+ (x A^T) B^T).
* grouped: row i of expert e (offsets[e] <= i < offsets[e + 1]) uses W_e and
  bias_e and row row_index[i] of x (a row of zeros for an index outside x).
* route: the k largest logits of a token, equal ones by lower expert, masked
  (-inf, NaN) ones never; softmax weights; rows sorted by expert, then token.
* combine: y[t] = residual[t] + sum_j weight[t, j] z[slot[t, j]].
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])

# Largest slope of each activation (the derivative's maximum over all v): GELU and
# its tanh form peak near v = sqrt(2) at 1.129 and 1.130, SiLU near 2.4 at 1.100.
SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "gelu_tanh": 1.131, "silu": 1.1}


def activate(name: str, v: np.ndarray) -> np.ndarray:
    v = np.asarray(v, np.float64)
    if name == "none":
        return v
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "gelu":
        return v * (1.0 + _erf(v / math.sqrt(2.0))) / 2.0
    if name == "gelu_tanh":
        return v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))) / 2.0
    if name == "silu":
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-v))
    raise ValueError(name)


def epilogue(z, act="none", gated=False, bias=None, gate=None, residual=None) -> np.ndarray:
    v = np.asarray(z, np.float64)
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    if gated:
        n = v.shape[1] // 2
        y = activate(act, v[:, :n]) * v[:, n:]
    else:
        y = activate(act, v)
    if gate is not None:
        y = y * np.asarray(gate, np.float64)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y


def grouped_products(x, weights, offsets, row_index=None) -> np.ndarray:
    """z [R, N] of float64 x [x_rows, K] and weights [E, N, K]; NaN in rows that no expert has."""
    rows = len(x) if row_index is None else len(row_index)
    z = np.full((rows, weights.shape[1]), np.nan)
    for e in range(weights.shape[0]):
        for i in range(offsets[e], offsets[e + 1]):
            src = i if row_index is None else int(row_index[i])
            xi = x[src] if 0 <= src < len(x) else np.zeros(x.shape[1])
            z[i] = weights[e] @ xi
    return z


def route(logits: np.ndarray, k: int, renormalize: bool):
    """(expert, weight, offsets, row_token, slot) as q2_route gives them, weights in float64."""
    logits = np.asarray(logits, np.float64)
    t, e = logits.shape
    expert = np.full((t, k), -1, np.int32)
    weight = np.zeros((t, k))
    for i in range(t):
        live = [j for j in range(e) if logits[i, j] > -math.inf]           # NaN compares false
        order = sorted(live, key=lambda j: (-logits[i, j], j))[:k]
        if not order:
            continue
        top = logits[i, order[0]]
        p = {j: 1.0 if logits[i, j] == top else math.exp(logits[i, j] - top) for j in live}
        total = sum(p[j] for j in (order if renormalize else live))
        for c, j in enumerate(order):
            expert[i, c] = j
            weight[i, c] = p[j] / total
    offsets = np.zeros(e + 1, np.int32)
    row_token = np.full(t * k, -1, np.int32)
    slot = np.full((t, k), -1, np.int32)
    row = 0
    for j in range(e):
        offsets[j] = row
        for i in range(t):
            for c in range(k):
                if expert[i, c] == j:
                    row_token[row] = i
                    slot[i, c] = row
                    row += 1
    offsets[e] = row
    return expert, weight, offsets, row_token, slot


def combine(z, slot, weight, residual=None) -> np.ndarray:
    t, k = slot.shape
    y = np.zeros((t, z.shape[1]))
    for i in range(t):
        for c in range(k):
            if 0 <= slot[i, c] < len(z):
                y[i] += float(weight[i, c]) * np.asarray(z[slot[i, c]], np.float64)
        if residual is not None:
            y[i] += np.asarray(residual[i], np.float64)
    return y
