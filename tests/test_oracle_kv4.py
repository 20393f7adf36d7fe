"""Pins of the 4-bit cache's oracle: the format by hand-placed nibbles, the quantiser by its extremes, its
ties and its half-step bound, eviction by hand-worked rows."""
import numpy as np
import pytest

from oracle import decoder as od
from oracle import kv4


@pytest.mark.parametrize("d", [64, 128])
def test_nibbles_by_hand(d):
    nb = d // 32
    for dim, key_at, val_at in ((0, 0, 0), (1, 1, 1), (9, nb * 8 + 1, 2 * nb * 4 + 1), (32 + 7, 8 + 7, nb * 4 + 4 + 3),
                                (31, 3 * nb * 8 + 7, 7 * nb * 4 + 3)):
        c = np.zeros(d, np.uint8)
        c[dim] = 11
        for key, at in ((True, key_at), (False, val_at)):
            row = kv4.pack_rows(c, key)
            assert row[at // 2] == 11 << (4 * (at % 2)) and np.count_nonzero(row) == 1, (dim, key)
    c = np.random.default_rng(d).integers(0, 16, (3, 5, d), dtype=np.uint8)
    for key in (True, False):
        assert np.array_equal(kv4.unpack_rows(kv4.pack_rows(c, key), key), c)


@pytest.mark.parametrize("g", [32, 64, 128])
def test_quantiser_extremes_constants_ties(g):
    x = np.zeros((4, 128), np.float32)
    x[0] = np.tile(np.arange(16, dtype=np.float32), 8) * 0.25 - 1.0       # every code, exactly
    x[1] = 3.0                                                            # constant
    x[2] = np.tile(np.array([0, 15, 0.5, 1.5, 2.5, 14.5, 7.5, 8.5], np.float32), 16)   # s = 1: ties to even
    x[3, 5] = np.inf
    c, sb, zb = kv4.quantize(x, g)
    v = kv4.dequantize(c, sb, zb)
    assert np.array_equal(v[0], x[0]) and np.array_equal(v[1], x[1])
    assert c[2, :8].tolist() == [0, 15, 0, 2, 2, 14, 8, 8]
    assert np.isnan(v[3, :g]).all() and (v[3, g:] == 0).all()


def test_quantiser_half_step():
    r = np.random.default_rng(1)
    x = (r.standard_normal((50, 128)) * np.exp(r.standard_normal((50, 1)) * 3) + r.standard_normal((50, 1))).astype(np.float32)
    for g in (32, 64, 128):
        c, sb, zb = kv4.quantize(x, g)
        s = np.repeat(kv4.bf16_value(sb), g, -1).astype(np.float64)
        z = np.repeat(kv4.bf16_value(zb), g, -1).astype(np.float64)
        # half a step; at the ends also the rounding of s (15 steps of 2^-9 each, a little more for the
        # single-precision quotient) and of z (2^-9 of |lo|)
        off = np.abs(kv4.dequantize(c, sb, zb) - x)
        assert (off <= s * (0.5 + 15 * 2.0 ** -9 * 1.01) + np.abs(z) * 2.0 ** -8).all()


def test_norm_rope_equals_the_step_oracle():
    r = np.random.default_rng(2)
    for d, sec in ((64, (8, 12, 12)), (128, (16, 24, 24))):
        x = r.standard_normal(d)
        pos = (7, 300, 41)
        mine = kv4.norm_rope(x, None, pos, 1e-6, 1e6, sec)
        ref = od.mrope(x[None, :], pos, d, 1e6, sec)[0]
        assert np.allclose(mine, ref, rtol=0, atol=1e-12)


def test_attention_by_hand():
    q = np.array([[1.0, 0.0], [0.0, 2.0]])
    K = np.array([[[0.0, 0.0], [np.log(3.0), 0.0]]])
    V = np.array([[[1.0, 0.0], [0.0, 1.0]]])
    out, mass = kv4.attention(q, K, V, 1.0)
    assert np.allclose(out, [[0.25, 0.75], [0.5, 0.5]]) and np.allclose(mass, [[0.75, 1.25]])
    out, mass = kv4.attention(q, K[:, :1], V[:, :1], 1.0)                  # one position: its V, weight 1 per head
    assert np.allclose(out, [[1, 0], [1, 0]]) and np.allclose(mass, [[2.0]])


def test_evict_by_hand():
    m = np.array([5.0, 1.0, 9.0, 1.0, 7.0, 0.0, 0.0])
    assert kv4.evict_positions(m, 7, 4, 2) == [2, 4, 5, 6]
    assert kv4.evict_positions(m, 7, 4, 0) == [0, 1, 2, 4]                  # of the two ones, the lower
    assert kv4.evict_positions(m, 7, 7, 3) == list(range(7))
    assert kv4.evict_positions(m, 3, 5, 5) == [0, 1, 2]
    assert kv4.evict_positions(m, 0, 5, 1) == []
    assert kv4.evict_positions(m, 7, 3, 3) == [4, 5, 6]
    assert kv4.evict_positions(np.array([np.nan, -1.0, -np.inf, 0.0]), 4, 3, 0) == [1, 2, 3]
    assert kv4.evict_positions(np.array([-0.0, 0.0, 1.0]), 3, 2, 0) == [0, 2]
