"""Plain CPU oracle of the products whose weights each token chooses.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports, links or executes this file; only tests do.  It shares
no code with the CUDA path: the router, the experts and the adapters are written from their definitions in numpy
float64, token by token.

Pinned in tests/test_oracle_moe.py: hand-worked choices and weights, experts of zero and constant weights, adapters
as a dense matrix.
"""
from __future__ import annotations

import numpy as np

__all__ = ["route", "dense", "experts", "adapters"]


def route(logits: np.ndarray, k: int, renorm: bool):
    """[T, E] -> ids int32 [T, k] and weights float64 [T, k]."""
    T, E = logits.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        row = [float(v) for v in logits[t]]
        live = [i for i in range(E) if row[i] > -np.inf]              # neither masked nor NaN
        order = sorted(live, key=lambda i: (-row[i], i))[:k]
        if not order:
            continue
        top = row[order[0]]
        p = {i: (1.0 if row[i] == top else float(np.exp(row[i] - top))) for i in live}
        total = sum(p[i] for i in (order if renorm else live))
        ids[t, :len(order)] = order
        w[t, :len(order)] = [p[i] / total for i in order]
    return ids, w


def dense(q: np.ndarray, s: np.ndarray, z: np.ndarray) -> np.ndarray:
    """Codes [N, K], scales and zeros [N, K / g] -> float64 [N, K]."""
    g = q.shape[-1] // s.shape[-1]
    return (q.astype(np.float64) - 8) * np.repeat(s.astype(np.float64), g, -1) + np.repeat(z.astype(np.float64), g, -1)


def experts(x, ids, weights, gate_up, down) -> np.ndarray:
    """x [T, H]; gate_up [E] of [2 I, H], down [E] of [H, I] -> [T, H]."""
    x = np.asarray(x, np.float64)
    y = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0 or e >= len(gate_up):
                continue
            h = gate_up[e] @ x[t]
            n = len(h) // 2
            with np.errstate(over="ignore"):
                act = h[:n] / (1.0 + np.exp(-h[:n])) * h[n:]
            y[t] += float(weights[t, j]) * (down[e] @ act)
    return y


def adapters(x, base, ids, a, b, ranks, scales) -> np.ndarray:
    """base [T, N] + scale B (A x); a [L, r, K], b [L, N, r]; ranks and scales per adapter."""
    y = np.array(base, np.float64)
    for t in range(x.shape[0]):
        i = int(ids[t])
        if 0 <= i < a.shape[0]:
            r = int(np.clip(ranks[i], 0, a.shape[1]))
            v = a[i, :r].astype(np.float64) @ np.asarray(x[t], np.float64)
            y[t] += float(scales[i]) * (b[i, :, :r].astype(np.float64) @ v)
    return y
