"""Plain CPU oracle of the 4-bit KV cache.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports, links or executes this file; only
tests do.  It shares no code with the CUDA path: the format is written from its specification in the
C header, attention and eviction from their definitions, in numpy float64 and plain loops.

A cached vector of d dims holds codes c in 0..15 and, per group of g dims, bf16 s and z:
value = c s + z.  The quantiser is defined on single-precision inputs with its roundings spelled out
(s = bf16(fl32((hi - lo) / 15)), z = bf16(lo), c = half-even rounding of (x - z) / s), so codes are
compared bit for bit; (x - z) / s is formed in float64 from the single-precision difference, which
cannot move a quotient of single-precision numbers across a rounding border of the code.

Pinned in tests/test_oracle_kv4.py: hand-placed nibbles, extremes that are hit exactly, constant
groups, the error bound of a half step, ties to even, and eviction against hand-worked rows.
"""
from __future__ import annotations

import numpy as np

__all__ = ["bf16_bits", "bf16_value", "quantize", "dequantize", "pack_rows", "unpack_rows", "pack_words",
           "norm_rope", "attention", "evict_positions"]


def bf16_bits(x) -> np.ndarray:
    """Bit patterns of x (float32) rounded to bf16, to nearest, ties to even; NaN becomes 0x7FC0."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16)).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32)


def quantize(x: np.ndarray, g: int):
    """float32 [..., d] -> codes uint8 [..., d], s bits and z bits uint16 [..., d / g]."""
    x = np.asarray(x, np.float32)
    y = x.reshape(*x.shape[:-1], x.shape[-1] // g, g)
    with np.errstate(all="ignore"):
        lo, hi = y.min(-1), y.max(-1)
        sb = bf16_bits((hi - lo) / np.float32(15))
        sb = np.where(sb < 0x0080, np.uint16(0), sb)
        zb = bf16_bits(lo)
        bad = ~np.isfinite(y).all(-1) | (sb >= 0x7F80) | ((zb & 0x7F80) == 0x7F80)
        sb, zb = np.where(bad, np.uint16(0), sb), np.where(bad, np.uint16(0x7FC0), zb)
        s, z = bf16_value(sb)[..., None], bf16_value(zb)[..., None]
        quo = (y - z).astype(np.float64) / np.where(s > 0, s, np.float32(1))
        c = np.where(s > 0, np.clip(np.rint(quo), 0, 15), 0)
    c = np.nan_to_num(c, nan=0.0).astype(np.uint8).reshape(x.shape)
    return c, sb, zb


def dequantize(c: np.ndarray, sb: np.ndarray, zb: np.ndarray) -> np.ndarray:
    g = c.shape[-1] // sb.shape[-1]
    y = c.reshape(*c.shape[:-1], c.shape[-1] // g, g).astype(np.float64)
    return (y * bf16_value(sb)[..., None].astype(np.float64) + bf16_value(zb)[..., None]).reshape(c.shape)


def _nibble(dim: int, d: int, key: bool) -> int:
    """Nibble index of a dim within its row: K [4][nb][8], V [8][nb][4]."""
    nb, b, r = d // 32, dim // 32, dim % 32
    return ((r // 8) * nb + b) * 8 + r % 8 if key else ((r // 4) * nb + b) * 4 + r % 4


def pack_rows(c: np.ndarray, key: bool) -> np.ndarray:
    d = c.shape[-1]
    out = np.zeros(c.shape[:-1] + (d // 2,), np.uint8)
    for dim in range(d):
        n = _nibble(dim, d, key)
        out[..., n // 2] |= (c[..., dim] << (4 * (n % 2))).astype(np.uint8)
    return out


def unpack_rows(b: np.ndarray, key: bool) -> np.ndarray:
    d = b.shape[-1] * 2
    out = np.zeros(b.shape[:-1] + (d,), np.uint8)
    for dim in range(d):
        n = _nibble(dim, d, key)
        out[..., dim] = (b[..., n // 2] >> (4 * (n % 2))) & 15
    return out


def pack_words(sb: np.ndarray, zb: np.ndarray) -> np.ndarray:
    return (zb.astype(np.uint32) | (sb.astype(np.uint32) << np.uint32(16))).view(np.int32)


def norm_rope(x: np.ndarray, w, pos3, eps: float, theta: float, sections) -> np.ndarray:
    """One head [d]: RMSNorm (w: float values or None), then the 3-section rotation of pairs (i, i + d/2)."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    if w is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * np.asarray(w, np.float64)
    out = np.empty(d)
    for i in range(d // 2):
        axis = 0 if i < sections[0] else (1 if i < sections[0] + sections[1] else 2)
        a = float(pos3[axis]) * float(theta) ** (-2.0 * i / d)
        out[i] = x[i] * np.cos(a) - x[i + d // 2] * np.sin(a)
        out[i + d // 2] = x[i + d // 2] * np.cos(a) + x[i] * np.sin(a)
    return out


def attention(q: np.ndarray, K: np.ndarray, V: np.ndarray, scale: float):
    """q [n_q, d], K and V [n_kv, L, d] -> out [n_q, d], and each position's weight summed over the query
    heads of its KV head [n_kv, L]."""
    nq, nkv = q.shape[0], K.shape[0]
    out, mass = np.zeros(q.shape), np.zeros(K.shape[:2])
    for i in range(nq):
        h = i // (nq // nkv)
        a = K[h] @ np.asarray(q[i], np.float64) * scale
        p = np.exp(a - a.max())
        p /= p.sum()
        out[i] = p @ V[h]
        mass[h] += p
    return out, mass


def evict_positions(mass: np.ndarray, n: int, keep: int, recent: int) -> list:
    """Positions of one (row, head) that stay, ascending: the newest, then the heaviest older ones."""
    total = min(n, keep)
    newest = min(recent, total)
    old = n - newest
    weight = [-np.inf if np.isnan(m) else float(m) for m in mass[:old]]
    nan = [bool(np.isnan(m)) for m in mass[:old]]
    order = sorted(range(old), key=lambda i: (nan[i], -weight[i], i))
    return sorted(order[:total - newest]) + list(range(old, n))
