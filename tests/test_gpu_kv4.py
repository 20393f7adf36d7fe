"""GPU parity of the 4-bit KV cache against its oracle: appended tokens, conversions, decode attention with
the mass, eviction, and a run of them together."""
import math

import numpy as np
import pytest

from gpu_helpers import rel_l2, require_gpu
import int4_weight_only_group_gb300 as kmr
from oracle import kv4

pytestmark = pytest.mark.gpu

SECTIONS = {64: (8, 12, 12), 128: (16, 24, 24)}
# fp32 scores: |error| <= (d + 4) 2^-24 sum|q k| scale, and with unit-variance q and k of 128 dims the sum is
# about 0.64 * 128 * 128^-0.5 = 7, so a weight is off by at most 5e-5 of itself, and so is an output
ATTN_TOL = 1e-4


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


def i32(torch, a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Cache:
    """A device cache and, beside it, the bf16-free truth: what each written position reads back as."""

    def __init__(self, torch, r, slots, nkv, S, d, g, fill=None, shift=0.0, spread=1.0):
        """fill: positions written per slot; the rest holds random codes with NaN scales."""
        self.torch, self.shape = torch, (slots, nkv, S, d, g)
        self.val, t = {}, {}
        for key in ("k", "v"):
            x = (r.standard_normal((slots, nkv, S, d)) * spread + shift).astype(np.float32)
            c, sb, zb = kv4.quantize(x, g)
            words = kv4.pack_words(sb, zb)
            rows = kv4.pack_rows(c, key == "k")
            self.val[key] = kv4.dequantize(c, sb, zb)
            if fill is not None:
                for s, n in enumerate(fill):
                    rows[s, :, n:] = r.integers(0, 256, rows[s, :, n:].shape, dtype=np.uint8)
                    words[s, :, n:] = kv4.pack_words(np.uint16([0x7FC0]), np.uint16([0x7FC0]))
            t[key], t[key + "w"] = torch.from_numpy(rows).cuda(), torch.from_numpy(words).cuda()
        self.dev = kmr.Kv4Cache(t["k"], t["v"], t["kw"], t["vw"])

    def host(self):
        return [t.cpu().numpy() for t in self.dev.tensors]


def attend(torch, cache, q, ids, cpos, mass=None, stream=None, scale=None):
    B, nq, d = q.shape
    n = kmr.kmr_decode_attn_kv4_workspace_size(cache, B, nq, mass is not None)
    assert n > 0
    ws = torch.full((n // 4,), float("nan"), device="cuda")
    out = torch.full((B, nq, d), float("nan"), device="cuda")
    kmr.kmr_decode_attn_kv4(cache, torch.from_numpy(q).cuda(), i32(torch, ids), i32(torch, cpos), B, nq,
                            scale or 1.0 / math.sqrt(d), mass, out, ws, n, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    return out.cpu().numpy()


# ------------------------------------------------------------------ conversion
@pytest.mark.parametrize("d,g", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64)])
def test_from_and_to_bf16_bit_exact(torch, d, g):
    """Spans of several lengths (0 and 1 among them), at odd starts, into scattered slots: the codes and scales
    are the oracle's bit for bit, everything outside the spans keeps its bits, and the way back gives
    bf16(c s + z)."""
    r = np.random.default_rng(d + g)
    nkv, S, S16, slots, slots16 = 3, 96, 77, 5, 4
    n, start, start16, ids, ids16 = [0, 1, 33, 75], [5, 95, 17, 0], [70, 3, 11, 2], [4, 0, 2, 3], [0, 1, 3, 2]
    x = [(r.standard_normal((slots16, nkv, S16, d)) * np.exp(r.standard_normal((slots16, nkv, S16, 1)))).astype(np.float32)
         for _ in range(2)]
    x[0][3, 0, 11] = 0.0                          # a constant row, ties, an infinity, a NaN, tiny and huge values
    x[0][3, 1, 12] = np.tile(np.float32([0, 15, 0.5, 1.5]), d // 4)
    x[1][3, 0, 13, 7] = np.inf
    x[1][3, 0, 14, 9] = np.nan
    x[1][3, 2, 15] *= np.float32(1e-38)
    x[0][3, 2, 16] *= np.float32(1e30)
    x[0][3, 2, 17, :2] = [3e38, -3e38]
    bits = [kv4.bf16_bits(a) for a in x]
    dev16 = [torch.from_numpy(b.view(np.int16)).cuda() for b in bits]
    c = Cache(torch, r, slots, nkv, S, d, g)
    before = c.host()
    args = [i32(torch, a) for a in (ids16, start16, ids, start, n)]
    kmr.kmr_kv4_from_bf16(c.dev, *dev16, slots16, S16, *args, 4, 80, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    want = [a.copy() for a in before]
    for b in range(4):
        for i, key in ((0, True), (1, False)):
            codes, sb, zb = kv4.quantize(kv4.bf16_value(bits[i][ids16[b], :, start16[b]:start16[b] + n[b]]), g)
            want[i][ids[b], :, start[b]:start[b] + n[b]] = kv4.pack_rows(codes, key)
            want[2 + i][ids[b], :, start[b]:start[b] + n[b]] = kv4.pack_words(sb, zb)
    for got, w in zip(c.host(), want):
        assert np.array_equal(got, w)
    back = [torch.full((slots16, nkv, S16, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kmr.kmr_kv4_to_bf16(c.dev, *back, slots16, S16, *args, 4, 80, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    for i in range(2):
        expect = np.full((slots16, nkv, S16, d), 7.0, np.float32)
        for b in range(4):
            at = (ids16[b], slice(None), slice(start16[b], start16[b] + n[b]))
            val = kv4.dequantize(*kv4.quantize(kv4.bf16_value(bits[i][at]), g))
            with np.errstate(all="ignore"):
                expect[at] = kv4.bf16_value(kv4.bf16_bits(val.astype(np.float32)))
        assert np.array_equal(back[i].float().cpu().numpy(), expect, equal_nan=True)


def test_convert_bad_and_clashing_spans(torch):
    r = np.random.default_rng(3)
    nkv, S, d, g, B = 2, 32, 64, 32, 6
    src = [torch.from_numpy(kv4.bf16_bits(r.standard_normal((B, nkv, S, d)).astype(np.float32)).view(np.int16)).cuda()
           for _ in range(2)]
    c = Cache(torch, r, 3, nkv, S, d, g)
    before = c.host()
    # rows 0..3 are bad: length, slot, end of the 4-bit row, end of the bf16 row; 4 and 5 overlap at 8..11
    ids, start, n = [0, 3, 0, 0, 1, 1], [0, 0, 30, 0, 4, 8], [17, 4, 4, 4, 8, 8]
    ids16, start16 = [0, 1, 2, 3, 4, 5], [0, 0, 0, 30, 0, 0]
    kmr.kmr_kv4_from_bf16(c.dev, *src, B, S, i32(torch, ids16), i32(torch, start16), i32(torch, ids), i32(torch, start),
                          i32(torch, n), B, 16, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() in (kmr.KMR_ERR_INVALID_ARG, kmr.KMR_ERR_SLOT_RANGE, kmr.KMR_ERR_CACHE_FULL)
    assert kmr.kmr_last_device_error() == 0
    after = c.host()
    for a, b in zip(after, before):
        assert np.array_equal(a[[0, 2]], b[[0, 2]]) and np.array_equal(a[1, :, :4], b[1, :, :4])
    x = kv4.bf16_value(src[0].cpu().numpy().view(np.uint16))
    for lo, hi, row, at in ((4, 8, 4, 0), (8, 16, 5, 0)):
        codes, sb, zb = kv4.quantize(x[row, :, at:at + hi - lo], g)
        assert np.array_equal(after[0][1, :, lo:hi], kv4.pack_rows(codes, True))
        assert np.array_equal(after[2][1, :, lo:hi], kv4.pack_words(sb, zb))
    # back: two spans onto one bf16 row
    dst = [torch.zeros((1, nkv, S, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    z = i32(torch, [0, 0])
    kmr.kmr_kv4_to_bf16(c.dev, *dst, 1, S, z, z, i32(torch, [0, 1]), i32(torch, [0, 4]), i32(torch, [8, 4]), 2, 8,
                        torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    first = kv4.dequantize(*kv4.quantize(x[4, :, 0:4], g)).astype(np.float32)
    assert np.array_equal(dst[0][0, :, :4].float().cpu().numpy(), kv4.bf16_value(kv4.bf16_bits(first)))
    assert bool((dst[0][0, :, 8:] == 0).all()) and bool((dst[0][0, :, 4:8] != 0).any())


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("d,g,nq,nkv,T", [(128, 32, 16, 8, 1), (64, 64, 4, 2, 5), (128, 128, 3, 3, 3), (64, 32, 8, 1, 17),
                                          (128, 64, 10, 5, 2), (64, 32, 7, 1, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_matches_oracle(torch, d, g, nq, nkv, T, norm):
    r = np.random.default_rng(d * g + nq + T)
    B, S, slots, theta, eps = 4, 64, 5, 1e6, 1e-6
    ids, cpos, n = [3, 0, 4, 1], [0, S - T, 20, 7], [T, T, max(0, T - 2), max(1, T // 2)]
    qkv = (r.standard_normal((B, T, nq + 2 * nkv, d)) * 3).astype(np.float32)
    pos = r.integers(-60, 200000, (3, B, T)).astype(np.int32)
    pos[:, 0] = pos[:1, 0]
    w = [1 + 0.1 * r.standard_normal(d).astype(np.float32) for _ in range(2)] if norm else [None, None]
    wb = [kv4.bf16_bits(a) if norm else None for a in w]
    c = Cache(torch, r, slots, nkv, S, d, g)
    before = c.host()
    q = torch.full((B, T, nq, d), 9.0, device="cuda")
    mass = torch.full((slots, nkv, S), 5.0, device="cuda")
    dev = [torch.from_numpy(a.view(np.int16)).cuda() if norm else None for a in wb]
    kmr.kmr_kv4_append(c.dev, torch.from_numpy(qkv).cuda(), torch.from_numpy(pos).cuda(), i32(torch, ids), i32(torch, cpos),
                       i32(torch, n), B, T, nq, dev[0], dev[1], eps, theta, SECTIONS[d], q, mass,
                       torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    got, kq = c.host(), q.cpu().numpy()
    mass = mass.cpu().numpy()
    touched = np.zeros((slots, S), bool)
    for b in range(B):
        assert (kq[b, n[b]:] == 9.0).all()
        for t in range(n[b]):
            at = cpos[b] + t
            touched[ids[b], at] = True
            assert (mass[ids[b], :, at] == 0).all()
            for h in range(nq + nkv):
                x = qkv[b, t, h]
                i = 0 if h < nq else 1
                want = kv4.norm_rope(x, kv4.bf16_value(wb[i]) if norm else None, pos[:, b, t], eps, theta, SECTIONS[d])
                plain = kv4.norm_rope(x, kv4.bf16_value(wb[i]) if norm else None, (0, 0, 0), eps, theta, SECTIONS[d])
                # about 16 roundings of 2^-24 (sum of squares, rsqrt, three products, cosine and sine, their
                # products and sum) of the pair's size
                size = np.abs(plain) + np.abs(np.roll(plain, d // 2))
                tol = 32 * 2.0 ** -24 * size
                if h < nq:
                    assert (np.abs(kq[b, t, h] - want) <= tol).all(), (b, t, h)
                else:
                    kvh = h - nq
                    codes = kv4.unpack_rows(got[0][ids[b], kvh, at], True)
                    u = got[2][ids[b], kvh, at].view(np.uint32)
                    sb, zb = (u >> 16).astype(np.uint16), (u & 0xFFFF).astype(np.uint16)
                    s, z = (np.repeat(kv4.bf16_value(a), g).astype(np.float64) for a in (sb, zb))
                    off = np.abs(kv4.dequantize(codes, sb, zb) - want)
                    assert (off <= s * (0.5 + 15 * 2.0 ** -9 * 1.01) + np.abs(z) * 2.0 ** -8 + tol).all()
            codes, sb, zb = kv4.quantize(qkv[b, t, nq + nkv:], g)              # V is quantised as it came
            assert np.array_equal(got[1][ids[b], :, at], kv4.pack_rows(codes, False))
            assert np.array_equal(got[3][ids[b], :, at], kv4.pack_words(sb, zb))
    for a, w0 in zip(got, before):
        for s in range(slots):
            assert np.array_equal(a[s][:, ~touched[s]], w0[s][:, ~touched[s]])
    assert all((mass[s][:, ~touched[s]] == 5.0).all() for s in range(slots))


def test_append_far_positions_keep_their_angle(torch):
    """Angles of positions near 2^31 (both signs): the fastest pair turns by a radian per position."""
    r = np.random.default_rng(8)
    d, nkv, nq, T = 128, 1, 1, 8
    pos1 = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -7, 0, 1, 999999937, -123456789], np.int64)
    pos = np.stack([pos1, pos1[::-1], np.roll(pos1, 3)])[:, None].astype(np.int32)
    qkv = r.standard_normal((1, T, 3, d)).astype(np.float32)
    c = kmr.Kv4Cache.zeros(1, nkv, 16, d, 32)
    q = torch.zeros((1, T, nq, d), device="cuda")
    kmr.kmr_kv4_append(c, torch.from_numpy(qkv).cuda(), torch.from_numpy(pos).cuda(), i32(torch, [0]), i32(torch, [0]),
                       None, 1, T, nq, None, None, 1e-6, 1e6, SECTIONS[d], q, None, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    for t in range(T):
        x = qkv[0, t, 0].astype(np.float64)
        want = np.empty(d)
        for i in range(d // 2):
            axis = 0 if i < 16 else (1 if i < 40 else 2)
            # in extended precision: a double's cosine at 2^31 radians is itself good to 2^-22 only in the frequency
            a = np.longdouble(int(pos[axis, 0, t])) * np.longdouble(1e6) ** (np.longdouble(-2 * i) / d)
            co, si = float(np.cos(a)), float(np.sin(a))
            want[i], want[i + 64] = x[i] * co - x[i + 64] * si, x[i + 64] * co + x[i] * si
        # the frequency in double (2^-53, 64 products) times 2^31 radians: 2^-53 * 64 * 2^31 = 2^-16 at worst,
        # and less the slower the pair; the roundings of the rotation beside it
        assert np.abs(q[0, t, 0].cpu().numpy() - want).max() <= 2.0 ** -16 * np.abs(x).max() * 2, t


def test_append_bad_and_clashing_rows(torch):
    r = np.random.default_rng(9)
    B, T, nq, nkv, d, g, S, slots = 7, 4, 2, 1, 64, 32, 32, 3
    qkv = r.standard_normal((B, T, nq + 2 * nkv, d)).astype(np.float32)
    #   bad: tokens -1, tokens 5, slot 3, slot -1, end; rows 5 and 6 overlap at positions 6, 7
    n, ids, cpos = [-1, 5, 4, 4, 4, 4, 4], [0, 0, 3, -1, 0, 1, 1], [0, 0, 0, 0, 29, 4, 6]
    c = Cache(torch, r, slots, nkv, S, d, g)
    before = c.host()
    q = torch.full((B, T, nq, d), 9.0, device="cuda")
    kmr.kmr_kv4_append(c.dev, torch.from_numpy(qkv).cuda(), torch.zeros((3, B, T), dtype=torch.int32, device="cuda"),
                       i32(torch, ids), i32(torch, cpos), i32(torch, n), B, T, nq, None, None, 1e-6, 1e6, SECTIONS[d], q,
                       None, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() in (kmr.KMR_ERR_INVALID_ARG, kmr.KMR_ERR_SLOT_RANGE, kmr.KMR_ERR_CACHE_FULL)
    got = c.host()
    assert (q[:5] == 9.0).all().item()
    assert np.array_equal(q[5:].cpu().numpy(), qkv[5:, :, :nq])          # position 0: no rotation; both rows' queries
    for a, w in zip(got, before):
        assert np.array_equal(a[[0, 2]], w[[0, 2]])
    for row, lo, hi in ((5, 4, 6), (6, 6, 10)):
        for i, off in ((0, nq), (1, nq + nkv)):
            codes, sb, zb = kv4.quantize(qkv[row, :hi - lo, off:off + nkv].transpose(1, 0, 2), g)
            assert np.array_equal(got[i][1, :, lo:hi], kv4.pack_rows(codes, i == 0)), (row, i)
            assert np.array_equal(got[2 + i][1, :, lo:hi], kv4.pack_words(sb, zb))


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("d,g", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64)])
@pytest.mark.parametrize("nq,nkv", [(16, 8), (4, 4), (8, 2), (3, 1), (5, 1), (16, 2), (7, 1)])
@pytest.mark.parametrize("S", [1104, 4112])                   # splits merged in a cluster, and through the workspace
def test_attention_matches_oracle(torch, d, g, nq, nkv, S):
    r = np.random.default_rng(d + g + nq)
    slots = 12
    L = [1, 2, 15, 16, 17, 127, 128, 129, 600, 1023, S]
    ids = [11, 3, 0, 5, 2, 7, 1, 9, 8, 10, 6]
    fill = [0] * slots
    for s, n in zip(ids, L):
        fill[s] = n
    c = Cache(torch, r, slots, nkv, S, d, g, fill)
    q = r.standard_normal((len(L), nq, d)).astype(np.float32) * 1.5
    mass0 = r.random((slots, nkv, S)).astype(np.float32)
    mass = torch.from_numpy(mass0.copy()).cuda()
    out = attend(torch, c.dev, q, ids, np.array(L) - 1, mass)
    assert kmr.kmr_last_device_error() == 0
    want = mass0.astype(np.float64)
    for b, n in enumerate(L):
        ref, m = kv4.attention(q[b], c.val["k"][ids[b], :, :n], c.val["v"][ids[b], :, :n], 1 / math.sqrt(d))
        assert rel_l2(out[b], ref) <= ATTN_TOL, (n, rel_l2(out[b], ref))
        want[ids[b], :, :n] += m
    got = mass.cpu().numpy()
    # a weight is off by ATTN_TOL of itself; the addition rounds once
    assert (np.abs(got - want) <= ATTN_TOL * (want - mass0) + 2.0 ** -23 * want).all()
    again = attend(torch, c.dev, q, ids, np.array(L) - 1)                  # without the mass: the same bits
    assert np.array_equal(out, again)
    for b in (0, 5, 10):                                                   # a row alone: the same bits
        one = attend(torch, c.dev, q[b:b + 1], ids[b:b + 1], [L[b] - 1])
        assert np.array_equal(one[0], out[b])


@pytest.mark.parametrize("L", [4095, 4096, 4097, 8191, 40000])
def test_attention_long_rows(torch, L):
    r = np.random.default_rng(L)
    S, nq, nkv, d, g = (L + 15) // 16 * 16, 4, 2, 128, 32
    c = Cache(torch, r, 1, nkv, S, d, g, [L])
    q = r.standard_normal((1, nq, d)).astype(np.float32) * 1.5
    mass = torch.zeros((1, nkv, S), device="cuda")
    out = attend(torch, c.dev, q, [0], [L - 1], mass)
    ref, m = kv4.attention(q[0], c.val["k"][0, :, :L], c.val["v"][0, :, :L], 1 / math.sqrt(d))
    assert rel_l2(out[0], ref) <= ATTN_TOL
    got = mass.cpu().numpy()[0]
    assert (got[:, L:] == 0).all() and (np.abs(got[:, :L] - m) <= ATTN_TOL * m + 1e-30).all()


@pytest.mark.parametrize("spread,shift", [(1e-4, 0.0), (1e4, 0.0), (1.0, 50.0), (3e6, 0.0), (1e-12, 0.0)])
@pytest.mark.parametrize("S", [512, 4112])
def test_attention_value_ranges(torch, spread, shift, S):
    """Values far from 1: the scales leave half precision's range on either side, or ride on a large base."""
    r = np.random.default_rng(17)
    L, nq, nkv, d, g = S - 12, 4, 2, 128, 32
    c = Cache(torch, r, 1, nkv, S, d, g, [L], shift, spread)
    # outlier groups among them: ranges that differ by 10^4 within a row
    q = (r.standard_normal((1, nq, d)) / max(spread, shift)).astype(np.float32)
    out = attend(torch, c.dev, q, [0], [L - 1])
    ref, _ = kv4.attention(q[0], c.val["k"][0, :, :L], c.val["v"][0, :, :L], 1 / math.sqrt(d))
    # with a base of 50 the scores are sums of 128 terms of about 0.8 each, as in ATTN_TOL's arithmetic
    assert rel_l2(out[0], ref) <= ATTN_TOL, rel_l2(out[0], ref)


def test_attention_scales_that_vary_along_the_row(torch):
    """A row whose values grow by 10^9 from first to last position, and one where they shrink: the early (late)
    positions are nothing beside the others, and neither overflow."""
    r = np.random.default_rng(18)
    S, nq, nkv, d, g = 1024, 2, 1, 64, 32
    for up in (True, False):
        c = Cache(torch, r, 1, nkv, S, d, g)
        ramp = np.exp(np.linspace(-10, 10, S) * (1 if up else -1))[None, :, None]
        x = (r.standard_normal((1, nkv, S, d)) * ramp).astype(np.float32)
        codes, sb, zb = kv4.quantize(x, g)
        c.dev.tensors[1].copy_(torch.from_numpy(kv4.pack_rows(codes, False)))
        c.dev.tensors[3].copy_(torch.from_numpy(kv4.pack_words(sb, zb)))
        q = r.standard_normal((1, nq, d)).astype(np.float32)
        out = attend(torch, c.dev, q, [0], [S - 1])
        ref, _ = kv4.attention(q[0], c.val["k"][0], kv4.dequantize(codes, sb, zb)[0], 1 / math.sqrt(d))
        assert rel_l2(out[0], ref) <= ATTN_TOL


def test_attention_sharp_and_flat_softmax(torch):
    """One position that takes all the weight (scores apart by hundreds), and q = 0: the mean of V."""
    r = np.random.default_rng(19)
    S, L, nq, nkv, d, g = 256, 201, 4, 2, 64, 64
    c = Cache(torch, r, 1, nkv, S, d, g, [L])
    q = np.zeros((1, nq, d), np.float32)
    out = attend(torch, c.dev, q, [0], [L - 1])
    mean = c.val["v"][0, :, :L].mean(1).repeat(nq // nkv, 0)
    assert np.abs(out[0] - mean).max() <= 2.0 ** -20
    q = np.stack([c.val["k"][0, h // 2, 77] * 40 for h in range(nq)])[None].astype(np.float32)
    out = attend(torch, c.dev, q, [0], [L - 1])
    # the weight is 1 to single precision; codes times scale and the base: three roundings
    assert np.abs(out[0] - c.val["v"][0, :, 77].repeat(nq // nkv, 0)).max() <= 2.0 ** -20


@pytest.mark.parametrize("S", [64, 4112])
def test_attention_bad_rows(torch, S):
    r = np.random.default_rng(20)
    nq, nkv, d, g, slots = 4, 2, 128, 64, 3
    c = Cache(torch, r, slots, nkv, S, d, g)
    q = r.standard_normal((6, nq, d)).astype(np.float32)
    mass = torch.zeros((slots, nkv, S), device="cuda")
    out = attend(torch, c.dev, q, [0, 3, -1, 1, 1, 2], [5, 5, 5, S, -1, S - 1], mass)
    assert kmr.kmr_last_device_error() in (kmr.KMR_ERR_SLOT_RANGE, kmr.KMR_ERR_CACHE_FULL)
    assert not out[1:5].any() and (mass[1] == 0).all().item()
    for b, s, n in ((0, 0, 6), (5, 2, S)):
        ref, m = kv4.attention(q[b], c.val["k"][s, :, :n], c.val["v"][s, :, :n], 1 / math.sqrt(d))
        assert rel_l2(out[b], ref) <= ATTN_TOL
        assert np.allclose(mass[s, :, :n].cpu().numpy(), m, rtol=2e-4, atol=0)


@pytest.mark.parametrize("S", [512, 4112])
def test_attention_rows_that_share_a_slot(torch, S):
    """Several rows of one slot (several continuations of a prompt): each attends on its own, and the slot's mass
    gains all of them, the same bits every run."""
    r = np.random.default_rng(21)
    nq, nkv, d, g = 4, 2, 128, 32
    c = Cache(torch, r, 2, nkv, S, d, g)
    ids, n = [1, 0, 1, 1, 0, 9], [300, 40, S, 7, 1, 5]
    q = r.standard_normal((6, nq, d)).astype(np.float32)
    runs = []
    for _ in range(3):
        mass = torch.zeros((2, nkv, S), device="cuda")
        out = attend(torch, c.dev, q, ids, np.array(n) - 1, mass)
        runs.append((out, mass.cpu().numpy()))
    assert all(np.array_equal(a, runs[0][0]) and np.array_equal(m, runs[0][1]) for a, m in runs)
    want = np.zeros((2, nkv, S))
    for b in range(5):
        ref, m = kv4.attention(q[b], c.val["k"][ids[b], :, :n[b]], c.val["v"][ids[b], :, :n[b]], 1 / math.sqrt(d))
        assert rel_l2(runs[0][0][b], ref) <= ATTN_TOL
        want[ids[b], :, :n[b]] += m
    assert (np.abs(runs[0][1] - want) <= (ATTN_TOL + 4 * 2.0 ** -24) * want).all()
    assert kmr.kmr_last_device_error() == kmr.KMR_ERR_SLOT_RANGE


def test_attention_beyond_32_bit_offsets(torch):
    """A slot whose codes start past 4 GB and whose elements pass 2^32."""
    r = np.random.default_rng(22)
    slots, nkv, S, d, g, L, nq = 9, 8, 1 << 20, 128, 128, 1000, 16
    tens = [torch.empty((slots, nkv, S, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    tens += [torch.empty((slots, nkv, S, d // g), dtype=torch.int32, device="cuda") for _ in range(2)]
    small = Cache(torch, r, 1, nkv, 1008, d, g)
    c = kmr.Kv4Cache(*tens)
    for t, s in zip(tens, small.dev.tensors):
        t[8, :, S - 1008:] = s[0]
    src = [torch.empty((1, nkv, 1008, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kmr.kmr_kv4_to_bf16(c, *src, 1, 1008, i32(torch, [0]), i32(torch, [0]), i32(torch, [8]), i32(torch, [S - 1008]),
                        i32(torch, [1008]), 1, 1008, torch.cuda.current_stream())
    kmr.kmr_kv4_from_bf16(c, *src, 1, 1008, i32(torch, [0]), i32(torch, [0]), i32(torch, [8]), i32(torch, [0]),
                          i32(torch, [1008]), 1, 1008, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    K, V = (a[0].float().cpu().numpy().astype(np.float64) for a in src)
    for i, x in ((0, K), (1, V)):
        codes, sb, zb = kv4.quantize(x, g)
        assert np.array_equal(tens[i][8, :, :1008].cpu().numpy(), kv4.pack_rows(codes, i == 0))
    vals = [kv4.dequantize(*kv4.quantize(x, g)) for x in (K, V)]
    q = r.standard_normal((1, nq, d)).astype(np.float32)
    out = attend(torch, c, q, [8], [L - 1])
    ref, _ = kv4.attention(q[0], vals[0][:, :L], vals[1][:, :L], 1 / math.sqrt(d))
    assert rel_l2(out[0], ref) <= ATTN_TOL


# ------------------------------------------------------------------ eviction
def evict(torch, src, dst, ids, dids, n, keep, recent, mass, dmass):
    B, nkv = len(ids), src.n_kv_heads
    kept = torch.full((B, nkv, keep), 77, dtype=torch.int32, device="cuda")
    new = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    kmr.kmr_kv4_evict(src, dst, i32(torch, ids), i32(torch, dids), i32(torch, n), B, keep, recent, mass, dmass, kept, new,
                      torch.cuda.current_stream())
    torch.cuda.synchronize()
    return kept.cpu().numpy(), new.cpu().numpy()


@pytest.mark.parametrize("d,g,nkv", [(128, 32, 8), (64, 64, 1), (128, 128, 2), (64, 32, 3)])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (17, 5), (64, 64), (300, 33), (512, 0)])
def test_evict_matches_oracle(torch, d, g, nkv, keep, recent):
    r = np.random.default_rng(d + keep)
    S, slots = 2064, 7
    n, ids, dids = [0, 1, 300, 301, 2064, 511, 2063], [6, 0, 3, 1, 2, 5, 4], [1, 0, 2, 6, 5, 3, 4]
    c = Cache(torch, r, slots, nkv, S, d, g)
    m = np.exp(2 * r.standard_normal((slots, nkv, S))).astype(np.float32)
    m[r.random(m.shape) < 0.3] = 0.0                        # ties at zero
    m[2, :, 100:1500] = np.float32(0.25)                    # a long run of equals
    m[5, 0, :200] = np.nan
    m[4, 0, 7], m[4, 0, 9], m[4, 0, 11] = np.inf, -np.inf, -0.0
    D = (keep + 15) // 16 * 16 + 16
    dst = Cache(torch, r, slots, nkv, D, d, g)
    before = dst.host()
    dm = torch.full((slots, nkv, D), 3.0, device="cuda")
    kept, new = evict(torch, c.dev, dst.dev, ids, dids, n, keep, recent, torch.from_numpy(m).cuda(), dm)
    assert kmr.kmr_last_device_error() == 0
    got, dm, srch = dst.host(), dm.cpu().numpy(), c.host()
    for b in range(len(n)):
        assert new[b] == min(n[b], keep)
        for h in range(nkv):
            want = kv4.evict_positions(m[ids[b], h], n[b], keep, recent)
            assert kept[b, h].tolist() == want + [-1] * (keep - len(want)), (b, h)
            for a, w0, s in zip(got, before, srch):
                assert np.array_equal(a[dids[b], h, :len(want)], s[ids[b], h, want])
                assert np.array_equal(a[dids[b], h, len(want):], w0[dids[b], h, len(want):])
            assert np.array_equal(dm[dids[b], h, :len(want)], m[ids[b], h, want], equal_nan=True)
            assert (dm[dids[b], h, len(want):] == 3.0).all()


@pytest.mark.parametrize("n", [60000, 131072])
def test_evict_long_rows(torch, n):
    r = np.random.default_rng(n)
    S, nkv, d, g, keep, recent = (n + 15) // 16 * 16, 2, 64, 64, 5000, 100
    src = kmr.Kv4Cache.zeros(1, nkv, S, d, g)
    src.tensors[0].random_(0, 256)
    m = np.exp(3 * r.standard_normal((1, nkv, S))).astype(np.float32)
    m = (np.round(m * 64) / 64).astype(np.float32)          # many ties
    dst = kmr.Kv4Cache.zeros(1, nkv, keep + 8, d, g)
    kept, new = evict(torch, src, dst, [0], [0], [n], keep, recent, torch.from_numpy(m).cuda(), None)
    assert kmr.kmr_last_device_error() == 0 and new.tolist() == [keep]
    for h in range(nkv):
        old = n - recent
        top = np.lexsort((np.arange(old), -m[0, h, :old]))[:keep - recent]
        want = np.concatenate([np.sort(top), np.arange(old, n)])
        assert np.array_equal(kept[0, h], want)
        assert np.array_equal(dst.tensors[0][0, h, :keep].cpu().numpy(), src.tensors[0][0, h].cpu().numpy()[want])


def test_evict_within_one_cache_and_refused_rows(torch):
    r = np.random.default_rng(31)
    slots, nkv, S, d, g, keep = 8, 2, 64, 64, 32, 10
    c = Cache(torch, r, slots, nkv, S, d, g)
    before = c.host()
    m = r.random((slots, nkv, S)).astype(np.float32)
    mass = torch.from_numpy(m.copy()).cuda()
    # row 0 is good (0 -> 7); 1: onto itself; 2 and 3: one destination; 4: onto row 0's source; 5: slot; 6: length
    ids, dids, n = [0, 1, 2, 3, 4, 8, 5], [7, 1, 6, 6, 0, 7 - 2, 3 + 0], [40, 20, 20, 20, 20, 20, 65]
    kept, new = evict(torch, c.dev, c.dev, ids, dids, n, keep, 3, mass, mass)
    assert kmr.kmr_last_device_error() in (kmr.KMR_ERR_SLOT_RANGE, kmr.KMR_ERR_CACHE_FULL)
    assert new.tolist() == [keep, 0, 0, 0, 0, 0, 0] and (kept[1:] == -1).all()
    got = c.host()
    for a, w in zip(got, before):
        assert np.array_equal(a[:7], w[:7])
        for h in range(nkv):
            want = kv4.evict_positions(m[0, h], 40, keep, 3)
            assert kept[0, h].tolist() == want
            assert np.array_equal(a[7, h, :keep], w[0, h, want]) and np.array_equal(a[7, h, keep:], w[7, h, keep:])
    gm = mass.cpu().numpy()
    assert np.array_equal(gm[:7], m[:7]) and np.array_equal(gm[7, 0, :keep], m[0, 0, kept[0, 0]])


# ------------------------------------------------------------------ together
def test_decode_evict_decode(torch):
    """As a program uses them: a prompt from a bf16 cache, tokens appended and attended with the mass gathered,
    the rows cut, and decoding going on in the cut rows; against the oracle's cache, step by step."""
    r = np.random.default_rng(41)
    B, nq, nkv, d, g, S, T0, eps, theta = 3, 4, 2, 128, 32, 128, 50, 1e-6, 1e6
    slots = 2 * B
    prompt = [kv4.bf16_bits(r.standard_normal((B, nkv, S, d)).astype(np.float32)) for _ in range(2)]
    lens = np.array([T0, T0 - 13, 1])
    cache = kmr.Kv4Cache.zeros(slots, nkv, S, d, g)
    st = torch.cuda.current_stream()
    ids, zero, rows = np.array([4, 1, 2]), i32(torch, [0] * B), i32(torch, range(B))
    kmr.kmr_kv4_from_bf16(cache, *[torch.from_numpy(p.view(np.int16)).cuda() for p in prompt], B, S, rows, zero,
                          i32(torch, ids), zero, i32(torch, lens), B, T0, st)
    K, V, M = {}, {}, {}
    for b in range(B):
        K[b], V[b] = (kv4.dequantize(*kv4.quantize(kv4.bf16_value(p[b, :, :lens[b]]), g)) for p in prompt)
        M[b] = np.zeros((nkv, lens[b]))
    mass = torch.zeros((slots, nkv, S), device="cuda")
    wb = [kv4.bf16_bits(1 + 0.1 * r.standard_normal(d).astype(np.float32)) for _ in range(2)]
    wdev = [torch.from_numpy(w.view(np.int16)).cuda() for w in wb]
    n_ws = kmr.kmr_decode_attn_kv4_workspace_size(cache, B, nq, True)
    ws = torch.empty(n_ws, dtype=torch.uint8, device="cuda")
    q, out = torch.zeros((B, 1, nq, d), device="cuda"), torch.zeros((B, nq, d), device="cuda")
    cur, pos0 = lens.copy(), lens + 100
    dslots = ids.copy()
    for step in range(24):
        if step == 16:
            keep, recent = 30, 8
            free = np.array([s for s in range(slots) if s not in dslots])[:B]
            kept, new = evict(torch, cache, cache, dslots, free, cur, keep, recent, mass, mass)
            mh = mass.cpu().numpy()
            for b in range(B):
                total = min(cur[b], keep)
                assert new[b] == total
                K2, V2, M2 = [], [], []
                for h in range(nkv):
                    # the device's own mass decides: two masses that differ by rounding may rank either way
                    want = kv4.evict_positions(mh[dslots[b], h], int(cur[b]), keep, recent)
                    assert kept[b, h, :total].tolist() == want
                    K2.append(K[b][h, want]), V2.append(V[b][h, want]), M2.append(M[b][h, want])
                K[b], V[b], M[b] = np.stack(K2), np.stack(V2), np.stack(M2)
            cur, dslots = new.astype(np.int64), free
        qkv = r.standard_normal((B, 1, nq + 2 * nkv, d)).astype(np.float32) * 2
        pos = np.stack([pos0 + step] * 3)[:, :, None].astype(np.int32)
        sl, cp = i32(torch, dslots), i32(torch, cur)
        kmr.kmr_kv4_append(cache, torch.from_numpy(qkv).cuda(), torch.from_numpy(pos).cuda(), sl, cp, None, B, 1, nq, *wdev,
                           eps, theta, SECTIONS[d], q, mass, st)
        kmr.kmr_decode_attn_kv4(cache, q, sl, cp, B, nq, 1 / math.sqrt(d), mass, out, ws, n_ws, st)
        assert kmr.kmr_last_device_error() == 0
        kc, vc, kw, vw = [t.cpu().numpy() for t in cache.tensors]
        got, mh = out.cpu().numpy(), mass.cpu().numpy()
        for b in range(B):
            at, s = int(cur[b]), dslots[b]
            rope = [kv4.norm_rope(qkv[b, 0, h], kv4.bf16_value(wb[0 if h < nq else 1]), pos[:, b, 0], eps, theta, SECTIONS[d])
                    for h in range(nq + nkv)]
            # the new key as the cache holds it (its codes may differ by one from the oracle's at a border)
            u = kw[s, :, at].view(np.uint32)
            kd = kv4.dequantize(kv4.unpack_rows(kc[s, :, at], True), (u >> 16).astype(np.uint16), (u & 0xFFFF).astype(np.uint16))
            assert rel_l2(kd, np.stack(rope[nq:])) <= 0.2
            vd = kv4.dequantize(*kv4.quantize(qkv[b, 0, nq + nkv:], g))
            K[b], V[b] = np.concatenate([K[b], kd[:, None]], 1), np.concatenate([V[b], vd[:, None]], 1)
            ref, m = kv4.attention(np.stack(rope[:nq]), K[b], V[b], 1 / math.sqrt(d))
            assert rel_l2(got[b], ref) <= 2 * ATTN_TOL, (step, b)
            M[b] = np.concatenate([M[b], np.zeros((nkv, 1))], 1) + m
            assert np.allclose(mh[s, :, :at + 1], M[b], rtol=1e-3, atol=1e-6)
        cur = cur + 1


def test_captured_and_replayed_on_another_stream(torch):
    """append + attention in one graph on a side stream: replays follow the state in place and equal eager calls."""
    r = np.random.default_rng(51)
    B, nq, nkv, d, g, S = 2, 16, 8, 128, 32, 256
    eager, graphed = (Cache(torch, np.random.default_rng(52), B, nkv, S, d, g, [100, 31]).dev for _ in range(2))
    n_ws = kmr.kmr_decode_attn_kv4_workspace_size(eager, B, nq, True)
    steps = [r.standard_normal((B, 1, nq + 2 * nkv, d)).astype(np.float32) for _ in range(4)]
    res = []
    side = torch.cuda.Stream()
    for cache, graph in ((eager, False), (graphed, True)):
        with torch.cuda.stream(side):
            qkv = torch.zeros((B, 1, (nq + 2 * nkv) * d), device="cuda")
            pos, cpos = torch.zeros((3, B, 1), dtype=torch.int32, device="cuda"), i32(torch, [100, 31])
            ids, ws = i32(torch, [0, 1]), torch.empty(n_ws, dtype=torch.uint8, device="cuda")
            q, out, mass = torch.zeros((B, 1, nq, d), device="cuda"), torch.zeros((B, nq, d), device="cuda"), torch.zeros((B, nkv, S), device="cuda")

            def one():
                st = torch.cuda.current_stream()
                kmr.kmr_kv4_append(cache, qkv, pos, ids, cpos, None, B, 1, nq, None, None, 1e-6, 1e6, SECTIONS[d], q, mass, st)
                kmr.kmr_decode_attn_kv4(cache, q, ids, cpos, B, nq, 1 / math.sqrt(d), mass, out, ws, n_ws, st)
                cpos.add_(1)
                pos.add_(1)

            if graph:
                kmr.kmr_last_device_error()
                G = torch.cuda.CUDAGraph()
                with torch.cuda.graph(G, stream=side):
                    one()
            got = []
            for x in steps:
                qkv.copy_(torch.from_numpy(x.reshape(B, 1, -1)))
                G.replay() if graph else one()
                got.append(out.clone())
            side.synchronize()
            res.append((torch.stack(got).cpu().numpy(), mass.cpu().numpy(), [t.cpu().numpy() for t in cache.tensors]))
    assert kmr.kmr_last_device_error() == 0
    assert np.array_equal(res[0][0], res[1][0]) and np.array_equal(res[0][1], res[1][1])
    for a, b in zip(res[0][2], res[1][2]):
        assert np.array_equal(a, b)


def test_two_streams_with_their_own_workspaces(torch):
    r = np.random.default_rng(61)
    S, nq, nkv, d, g, B = 2048, 16, 8, 128, 32, 4
    c = Cache(torch, r, B, nkv, S, d, g)
    q = torch.from_numpy(r.standard_normal((2, B, nq, d)).astype(np.float32)).cuda()
    ids, cpos = i32(torch, range(B)), i32(torch, [2047, 3, 700, 1500])
    n = kmr.kmr_decode_attn_kv4_workspace_size(c.dev, B, nq)
    out = torch.zeros((2, B, nq, d), device="cuda")
    ref = torch.zeros_like(out)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for i in range(2):
        kmr.kmr_decode_attn_kv4(c.dev, q[i], ids, cpos, B, nq, 0.08, None, ref[i], ws[0], n, torch.cuda.current_stream())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            kmr.kmr_decode_attn_kv4(c.dev, q[i], ids, cpos, B, nq, 0.08, None, out[i], ws[i], n, streams[i])
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


# ------------------------------------------------------------------ limits, leftovers, the framework's own cache
def test_shared_memory_leftovers_do_not_matter(torch):
    """Shared memory filled with NaN bits before every call: the same bits as without."""
    r = np.random.default_rng(71)
    for S, L, nq, nkv, d, g in ((1024, [1, 70, 129, 1000], 16, 8, 128, 32), (4112, [1, 70, 300, 4100], 8, 1, 64, 64)):
        c = Cache(torch, r, 4, nkv, S, d, g, L)
        q = r.standard_normal((4, nq, d)).astype(np.float32)
        res = []
        for poison in (None, 0xFFFFFFFF, 0x7F800000):
            mass = torch.zeros((4, nkv, S), device="cuda")
            if poison is not None:
                kmr.kmr_smem_poison(poison, torch.cuda.current_stream())
            out = attend(torch, c.dev, q, range(4), np.array(L) - 1, mass)
            if poison is not None:
                kmr.kmr_smem_poison(poison, torch.cuda.current_stream())
            dst = Cache(torch, np.random.default_rng(1), 4, nkv, 64, d, g)
            kept, new = evict(torch, c.dev, dst.dev, range(4), range(4), L, 50, 5, mass, None)
            res.append([out, mass.cpu().numpy(), kept, new] + dst.host())
        for other in res[1:]:
            assert all(np.array_equal(a, b) for a, b in zip(res[0], other))


@pytest.mark.parametrize("S", [16, 4112])
def test_the_most_rows(torch, S):
    """1024 rows in one call: appended, attended (a quarter of them sharing slots) and evicted."""
    r = np.random.default_rng(72)
    B, nq, nkv, d, g = 1024, 2, 1, 64, 64
    slots = 768
    ids = np.concatenate([np.arange(768), r.integers(0, 768, 256)])
    cache = kmr.Kv4Cache.zeros(slots, nkv, S, d, g)
    qkv = r.standard_normal((B, 1, nq + 2 * nkv, d)).astype(np.float32)
    q = torch.zeros((B, 1, nq, d), device="cuda")
    sl, zero = i32(torch, ids), i32(torch, [0] * B)
    kmr.kmr_kv4_append(cache, torch.from_numpy(qkv).cuda(), torch.zeros((3, B, 1), dtype=torch.int32, device="cuda"), sl, zero,
                       None, B, 1, nq, None, None, 1e-6, 1e6, SECTIONS[d], q, None, torch.cuda.current_stream())
    last = {s: b for b, s in enumerate(ids)}                          # the later row's token stays
    V = kv4.dequantize(*kv4.quantize(qkv[:, 0, nq + nkv:], g))
    mass = torch.zeros((slots, nkv, S), device="cuda")
    out = attend(torch, cache, q.cpu().numpy()[:, 0], ids, [0] * B, mass)
    want = np.stack([V[last[s]] for s in ids]).repeat(nq, 1)
    assert kmr.kmr_last_device_error() == 0
    # one position: weight 1, and a code times its scale plus a base
    assert np.abs(out - want).max() <= 2.0 ** -20
    m = mass.cpu().numpy()[:, 0, 0]
    assert np.array_equal(m, nq * np.bincount(ids, minlength=slots).astype(np.float32))
    dst = kmr.Kv4Cache.zeros(B, nkv, 16, d, g)
    kept, new = evict(torch, cache, dst, ids, np.arange(B)[::-1].copy(), [1] * B, 3, 1, mass, None)
    assert kmr.kmr_last_device_error() == 0
    assert (new == 1).all() and (kept[:, 0] == [0, -1, -1]).all()
    got = dst.tensors[1][:, 0, 0].cpu().numpy()[::-1]
    assert np.array_equal(got, cache.tensors[1][ids.tolist(), 0, 0].cpu().numpy())


def test_convert_long_spans(torch):
    """Many long spans (a CTA takes 256 positions), two of them onto the same positions of a slot."""
    r = np.random.default_rng(73)
    B, nkv, d, g, S = 16, 8, 128, 32, 1024
    x = r.standard_normal((2, B, nkv, S, d)).astype(np.float32)
    bits = kv4.bf16_bits(x)
    dev16 = [torch.from_numpy(b.view(np.int16)).cuda() for b in bits]
    cache = kmr.Kv4Cache.zeros(B, nkv, S, d, g)
    n = [1024, 1000, 257, 256, 255, 1, 0, 700] * 2
    ids = list(range(B))
    start = [0] * B
    ids[15], start[15] = 8, 324                                       # row 15: 324.. of row 8's slot, over its values
    rows, zero = i32(torch, range(B)), i32(torch, [0] * B)
    kmr.kmr_kv4_from_bf16(cache, *dev16, B, S, rows, zero, i32(torch, ids), i32(torch, start), i32(torch, n), B, S,
                          torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    for i in range(2):
        codes, sb, zb = kv4.quantize(kv4.bf16_value(bits[i]), g)
        want, words = np.zeros((B, nkv, S, d // 2), np.uint8), np.zeros((B, nkv, S, d // g), np.int32)
        for b in range(B):
            at = (ids[b], slice(None), slice(start[b], start[b] + n[b]))
            want[at], words[at] = kv4.pack_rows(codes[b, :, :n[b]], i == 0), kv4.pack_words(sb[b, :, :n[b]], zb[b, :, :n[b]])
        assert np.array_equal(cache.tensors[i].cpu().numpy(), want)
        assert np.array_equal(cache.tensors[2 + i].cpu().numpy(), words)
    back = [torch.zeros((B, nkv, S, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kmr.kmr_kv4_to_bf16(cache, *back, B, S, rows, zero, rows, zero, i32(torch, [S] * B), B, S, torch.cuda.current_stream())
    val = kv4.dequantize(kv4.unpack_rows(cache.tensors[0].cpu().numpy(), True), *(
        (cache.tensors[2].cpu().numpy().view(np.uint32) >> k).astype(np.uint16) for k in (16, 0)))
    assert np.array_equal(back[0].float().cpu().numpy(), kv4.bf16_value(kv4.bf16_bits(val.astype(np.float32))))


def test_poisoned_group_reaches_its_own_dims_only(torch):
    """An infinity in one position's V: NaN in that group's dims of the rows that attend it, nothing elsewhere."""
    r = np.random.default_rng(74)
    S, nq, nkv, d, g = 64, 2, 1, 128, 32
    x = r.standard_normal((2, 1, nkv, S, d)).astype(np.float32)
    x[1, 0, 0, 9, 40] = np.inf
    cache = kmr.Kv4Cache.zeros(1, nkv, S, d, g)
    z = i32(torch, [0])
    kmr.kmr_kv4_from_bf16(cache, *[torch.from_numpy(kv4.bf16_bits(a).view(np.int16)).cuda() for a in x], 1, S, z, z, z, z,
                          i32(torch, [S]), 1, S, torch.cuda.current_stream())
    q = r.standard_normal((2, nq, d)).astype(np.float32)
    out = attend(torch, cache, q, [0, 0], [8, 9])
    assert np.isfinite(out[0]).all()
    assert np.isnan(out[1][:, 32:64]).all() and np.isfinite(np.delete(out[1], range(32, 64), 1)).all()


def test_prefilled_model_cache_to_4_bits(torch):
    """kmr_prefill fills the model's bf16 cache; its rows go to 4 bits (kmr_model_kv_pointers) and are attended."""
    from gpu_helpers import d2h_bytes
    from int4_weight_only_group_gb300 import driver
    from workloads import SyntheticModel, tiny_workload
    wl = tiny_workload()
    cfg = wl.cfg
    m = kmr.Model.from_config(cfg, max_batch=1)
    driver.load_weights(m, SyntheticModel(cfg, wl.seed), cfg.n_layers, cfg.qk_norm)
    T, nkv, d, S = 40, cfg.n_kv_heads, cfg.head_dim, cfg.max_len
    m.reserve_prefill(T)
    r = np.random.default_rng(75)
    state = [torch.zeros(n, dtype=t, device="cuda") for n, t in ((1, torch.int32), (3, torch.int32), (1, torch.int32), (1, torch.uint8))]
    m.prefill(torch.from_numpy(r.integers(1, cfg.vocab - 1, T).astype(np.int32)).cuda(),
              torch.arange(T, dtype=torch.int32, device="cuda").repeat(3, 1).contiguous(), T, 0, 0, *state, None,
              torch.cuda.current_stream())
    assert m.sync_status() == 0
    z = i32(torch, [0])
    for layer in range(cfg.n_layers):
        cache = kmr.Kv4Cache.zeros(1, nkv, S, d, 32)
        kp, vp = m.kv_pointers(layer)
        kmr.kmr_kv4_from_bf16(cache, kp, vp, cfg.slots, S, z, z, z, z, i32(torch, [T]), 1, T, torch.cuda.current_stream())
        q = r.standard_normal((1, cfg.n_q_heads, d)).astype(np.float32)
        out = attend(torch, cache, q, [0], [T - 1])
        assert kmr.kmr_last_device_error() == 0
        K, V = (kv4.bf16_value(d2h_bytes(p, nkv * S * d * 2).view(np.uint16)).reshape(nkv, S, d)[:, :T] for p in (kp, vp))
        ref, _ = kv4.attention(q[0], *(kv4.dequantize(*kv4.quantize(a, 32)) for a in (K, V)), 1 / math.sqrt(d))
        assert rel_l2(out[0], ref) <= ATTN_TOL
    m.close()


def test_two_streams_long_rows(torch):
    r = np.random.default_rng(76)
    S, nq, nkv, d, g, B = 5008, 4, 2, 64, 32, 3
    c = Cache(torch, r, B, nkv, S, d, g)
    q = torch.from_numpy(r.standard_normal((2, B, nq, d)).astype(np.float32)).cuda()
    ids, cpos = i32(torch, range(B)), i32(torch, [5007, 3, 2700])
    n = kmr.kmr_decode_attn_kv4_workspace_size(c.dev, B, nq, True)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out, mass = torch.zeros((3, 2, B, nq, d), device="cuda"), torch.zeros((3, 2, B, nkv, S), device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for run in range(3):
        for i in range(2):
            kmr.kmr_decode_attn_kv4(c.dev, q[i], ids, cpos, B, nq, 0.1, mass[run, i], out[run, i], ws[i], n, streams[i])
        if run == 0:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out[1], out[0]) and torch.equal(out[2], out[0]) and torch.equal(mass[1], mass[0])
    for i in range(2):
        for b, L in enumerate((5008, 4, 2701)):
            ref, m = kv4.attention(q[i, b].cpu().numpy(), c.val["k"][b, :, :L], c.val["v"][b, :, :L], 0.1)
            assert rel_l2(out[0, i, b].cpu().numpy(), ref) <= ATTN_TOL
            assert np.allclose(mass[0, i, b, :, :L].cpu().numpy(), m, rtol=2e-4, atol=1e-30)


@pytest.mark.parametrize("S", [1024, 2048, 2064])
def test_a_row_s_bits_do_not_depend_on_the_batch(torch, S):
    """Few rows have a CTA for every split, many rows several splits a CTA: the same output and mass, bit for bit."""
    r = np.random.default_rng(S)
    nq, nkv, d, g, slots = 16, 8, 128, 32, 128
    L = r.integers(1, S + 1, slots)
    L[:4] = [S, S - 1, 129, 1]
    c = kmr.Kv4Cache.zeros(slots, nkv, S, d, g)
    for t in c.tensors[:2]:
        t.random_(0, 256)
    for t in c.tensors[2:]:                                           # scales of about 1/4, bases of about -2
        t.copy_(torch.from_numpy(kv4.pack_words(kv4.bf16_bits(r.uniform(0.2, 0.3, t.shape).astype(np.float32)),
                                                kv4.bf16_bits(r.uniform(-2.2, -1.8, t.shape).astype(np.float32)))))
    q = r.standard_normal((slots, nq, d)).astype(np.float32)
    res = []
    for B in (2, 16, 40, 128):
        mass = torch.zeros((slots, nkv, S), device="cuda")
        out = attend(torch, c, q[:B], range(B), L[:B] - 1, mass)
        plain = attend(torch, c, q[:B], range(B), L[:B] - 1)
        assert np.array_equal(out, plain)
        res.append((out, mass[:B].cpu().numpy()))
    assert kmr.kmr_last_device_error() == 0
    for out, mass in res[:-1]:
        assert np.array_equal(out, res[-1][0][:len(out)]) and np.array_equal(mass, res[-1][1][:len(out)])
    vals = [kv4.dequantize(kv4.unpack_rows(t[:3].cpu().numpy(), i == 0), *((w[:3].cpu().numpy().view(np.uint32) >> k).astype(np.uint16)
            for k in (16, 0))) for i, (t, w) in enumerate(zip(c.tensors[:2], c.tensors[2:]))]
    for b in range(3):
        ref, m = kv4.attention(q[b], vals[0][b, :, :L[b]], vals[1][b, :, :L[b]], 1 / math.sqrt(d))
        assert rel_l2(res[-1][0][b], ref) <= ATTN_TOL
        assert np.allclose(res[-1][1][b, :, :L[b]], m, rtol=2e-4, atol=1e-30)


@pytest.mark.parametrize("S", [64, 4112])
def test_idle_rows(torch, S):
    """A padded batch: idle rows (no token, position -1, length 0) with slots that are out of range or somebody
    else's change nothing and raise nothing."""
    r = np.random.default_rng(80)
    nq, nkv, d, g, slots = 2, 1, 64, 32, 3
    c = Cache(torch, r, slots, nkv, S, d, g)
    before = c.host()
    qkv = r.standard_normal((3, 1, nq + 2 * nkv, d)).astype(np.float32)
    qo = torch.full((3, 1, nq, d), 4.0, device="cuda")
    mass = torch.ones((slots, nkv, S), device="cuda")
    ids = [0, 99, 0]
    kmr.kmr_kv4_append(c.dev, torch.from_numpy(qkv).cuda(), torch.zeros((3, 3, 1), dtype=torch.int32, device="cuda"),
                       i32(torch, ids), i32(torch, [5, 5, 5]), i32(torch, [1, 0, 0]), 3, 1, nq, None, None, 1e-6, 1e6,
                       SECTIONS[d], qo, mass, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    assert (qo[1:] == 4.0).all().item() and mass[0, 0, 5].item() == 0 and mass.sum().item() == slots * S - 1
    got = c.host()
    for a, w in zip(got, before):
        assert np.array_equal(np.delete(a[0], 5, 1), np.delete(w[0], 5, 1)) and np.array_equal(a[1:], w[1:])
    q = r.standard_normal((3, nq, d)).astype(np.float32)
    mass.zero_()
    out = attend(torch, c.dev, q, ids, [5, -1, -1], mass)
    assert kmr.kmr_last_device_error() == 0
    one = torch.zeros_like(mass)
    alone = attend(torch, c.dev, q[:1], [0], [5], one)
    assert np.array_equal(out[0], alone[0]) and not out[1:].any() and torch.equal(mass, one)
    assert abs(mass.sum().item() - nq) <= 1e-5
    dst = Cache(torch, r, 2, nkv, 16, d, g)
    kept, new = evict(torch, c.dev, dst.dev, [0, 99, 0], [1, 1, -5], [6, 0, 0], 4, 1, mass, None)
    assert kmr.kmr_last_device_error() == 0
    assert new.tolist() == [4, 0, 0] and (kept[1:] == -1).all()
    assert kept[0, 0].tolist() == kv4.evict_positions(mass[0, 0].cpu().numpy(), 6, 4, 1)


FRESH = """
import math, sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import numpy as np, torch
import int4_weight_only_group_gb300 as kmr
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
one = kmr.Kv4Cache.zeros(1, 1, 16, 64, 32)
q0 = torch.zeros((1, 1, 1, 64), device="cuda")
kmr.kmr_kv4_append(one, torch.zeros((1, 1, 3, 64), device="cuda"), torch.zeros((3, 1, 1), dtype=torch.int32, device="cuda"),
                   i32([0]), i32([0]), None, 1, 1, 1, None, None, 1e-6, 1e6, (8, 12, 12), q0, None, torch.cuda.current_stream())
torch.cuda.synchronize()
for S in (256, 4112):
    B, nq, nkv, d, g = 2, 8, 2, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(S)
    src = [torch.randn((B, nkv, S, d), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    q = torch.randn((B, nq, d), generator=gen, device="cuda")
    rows, zero, n = i32([0, 1]), i32([0, 0]), i32([S, S - 9])
    res = []
    for captured in (True, False):
        c, dst = kmr.Kv4Cache.zeros(B, nkv, S, d, g), kmr.Kv4Cache.zeros(B, nkv, 64, d, g)
        mass, out = torch.zeros((B, nkv, S), device="cuda"), torch.zeros((B, nq, d), device="cuda")
        nb = kmr.kmr_decode_attn_kv4_workspace_size(c, B, nq, True)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        kept, new = torch.zeros((B, nkv, 50), dtype=torch.int32, device="cuda"), i32([0, 0])
        back = [torch.zeros((B, nkv, 64, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        last = n - 1
        def run():
            st = torch.cuda.current_stream()
            kmr.kmr_kv4_from_bf16(c, src[0], src[1], B, S, rows, zero, rows, zero, n, B, S, st)
            kmr.kmr_decode_attn_kv4(c, q, rows, last, B, nq, 1 / math.sqrt(d), mass, out, ws, nb, st)
            kmr.kmr_kv4_evict(c, dst, rows, rows, n, B, 50, 7, mass, None, kept, new, st)
            kmr.kmr_kv4_to_bf16(dst, back[0], back[1], B, 64, rows, zero, rows, zero, new, B, 50, st)
        if captured:
            G = torch.cuda.CUDAGraph()
            with torch.cuda.graph(G):
                run()
            G.replay()
        else:
            run()
        torch.cuda.synchronize()
        res.append([out, mass, kept, new] + back)
    assert all(torch.equal(a, b) for a, b in zip(*res)), S
    assert res[0][0].abs().sum().item() > 0 and int(res[0][3][0]) == 50
assert kmr.kmr_last_device_error() == 0
print("fresh ok")
"""


def test_first_calls_of_other_shapes_inside_a_capture(torch):
    """In a process whose only earlier call was another operator of another shape, every operator is captured and
    replayed: the same bits as eager calls."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH.replace("{root!r}", repr(root))], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fresh ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


# ------------------------------------------------------------------ values that the codes' scales do not reach alike
def set_values(torch, c, x, g):
    """The cache's V from x (float32 [slots, nkv, S, d]); returns what it reads back as."""
    codes, sb, zb = kv4.quantize(x, g)
    c.dev.tensors[1].copy_(torch.from_numpy(kv4.pack_rows(codes, False)))
    c.dev.tensors[3].copy_(torch.from_numpy(kv4.pack_words(sb, zb)))
    return kv4.dequantize(codes, sb, zb)


@pytest.mark.parametrize("d,g,nq,nkv,S,L", [(128, 32, 16, 8, 1104, 1100), (128, 32, 4, 1, 1104, 1100), (64, 32, 2, 1, 1104, 1100),
                                            (128, 128, 2, 1, 4112, 4100), (128, 32, 16, 8, 4112, 4100), (64, 64, 8, 1, 4112, 4100),
                                            (128, 64, 8, 1, 208, 200), (128, 32, 7, 1, 4112, 4100)])
def test_constant_values(torch, d, g, nq, nkv, S, L):
    """V constant over every group (scale 0): the output is the base, whatever the keys; with V = 0 it is 0.  Keys whose
    best score rises by a few octaves along the row, as random ones do."""
    r = np.random.default_rng(L + d + nq)
    c = Cache(torch, r, 1, nkv, S, d, g, [L])
    q = (r.standard_normal((1, nq, d)) * 3).astype(np.float32)
    for value in (1.0, 0.0, -3.5, None):
        x = np.full((1, nkv, S, d), value if value is not None else 0.0, np.float32)
        if value is None:                                    # a base of its own for every group
            x += np.repeat(np.arange(1, d // g + 1, dtype=np.float32) * [1, -2, 4, -8][:d // g], g)
        set_values(torch, c, x, g)
        out = attend(torch, c.dev, q, [0], [L - 1])
        # the weights' sum and the weights times the base: at most 128 roundings of 2^-24 in either
        want = x[0, 0, 0]
        assert (np.abs(out[0] - want) <= 256 * 2.0 ** -24 * np.abs(want)).all(), value
    assert kmr.kmr_last_device_error() == 0


@pytest.mark.parametrize("S,L", [(1104, 1100), (4112, 4100)])
def test_tiny_values(torch, S, L):
    """V of about 2^-118: what it adds to the weights' scaling stays finite."""
    r = np.random.default_rng(S)
    nq, nkv, d, g = 4, 2, 128, 32
    c = Cache(torch, r, 1, nkv, S, d, g, [L])
    V = set_values(torch, c, (r.standard_normal((1, nkv, S, d)) * 2.0 ** -118).astype(np.float32), g)
    q = (r.standard_normal((1, nq, d)) * 3).astype(np.float32)
    out = attend(torch, c.dev, q, [0], [L - 1])
    ref, _ = kv4.attention(q[0], c.val["k"][0, :, :L], V[0, :, :L], 1 / math.sqrt(d))
    # scales of about 2^-120: a weight below 2^-5 times one leaves the normal range, at 2^-149 of 2^-118 (the output is
    # some 2^-4 of V) 2^-27 each
    assert rel_l2(out[0].astype(np.float64) * 2.0 ** 118, ref * 2.0 ** 118) <= ATTN_TOL


# ------------------------------------------------------------------ refused rows claim nothing
@pytest.mark.parametrize("to_bf16", [False, True])
@pytest.mark.parametrize("T", [20, 300])                        # short and long spans of a CTA
def test_refused_later_spans_leave_the_earlier_ones_alone(torch, to_bf16, T):
    """Later rows that would write the same positions but are refused, each for another reason, those of the side
    that is only read among them: the good row's span is written whole."""
    r = np.random.default_rng(90 + T)
    nkv, d, g, S, slots = 16, 64, 32, 320, 3
    src = [torch.from_numpy(kv4.bf16_bits(r.standard_normal((slots, nkv, S, d)).astype(np.float32)).view(np.int16)).cuda()
           for _ in range(2)]
    c = Cache(torch, r, slots, nkv, S, d, g)
    big = 2 ** 31 - 1
    # (length, slot, start) of the written and of the read side
    bad = [(T, (1, 5), (7, 0)), (T, (1, 5), (-1, 0)), (T, (1, 5), (0, S - T + 1)), (T, (1, 5), (0, -1)), (T, (1, 5), (0, big)),
           (-1, (1, 5), (0, 0)), (T + 1, (1, 5), (0, 0)), (T, (1, S - T + 1), (0, 0)), (T, (1, -1), (0, 0)), (T, (1, big), (0, 0))]
    rows = [(T, (1, 5), (2, 3))] + bad
    n = i32(torch, [a[0] for a in rows])
    w, rd = ([i32(torch, [a[side][k] for a in rows]) for k in (0, 1)] for side in (1, 2))
    B, st = len(rows), torch.cuda.current_stream()
    if to_bf16:
        dst = [torch.zeros((slots, nkv, S, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        kmr.kmr_kv4_to_bf16(c.dev, *dst, slots, S, *w, *rd, n, B, T, st)
    else:
        kmr.kmr_kv4_from_bf16(c.dev, *src, slots, S, *rd, *w, n, B, T, st)
    assert kmr.kmr_last_device_error() in (kmr.KMR_ERR_INVALID_ARG, kmr.KMR_ERR_SLOT_RANGE, kmr.KMR_ERR_CACHE_FULL)
    for i, key in ((0, "k"), (1, "v")):
        if to_bf16:
            want = np.zeros((slots, nkv, S, d), np.float32)
            want[1, :, 5:5 + T] = kv4.bf16_value(kv4.bf16_bits(c.val[key][2, :, 3:3 + T].astype(np.float32)))
            assert np.array_equal(dst[i].float().cpu().numpy(), want)
        else:
            codes, sb, zb = kv4.quantize(kv4.bf16_value(src[i].cpu().numpy().view(np.uint16)[2, :, 3:3 + T]), g)
            got = c.host()
            assert np.array_equal(got[i][1, :, 5:5 + T], kv4.pack_rows(codes, key == "k"))
            assert np.array_equal(got[2 + i][1, :, 5:5 + T], kv4.pack_words(sb, zb))


# ------------------------------------------------------------------ groups and positions of very different scale
# Keys here give scores of a few units, off by some 20 roundings of partial sums of about 20 (base 2), 2^-25 of them each
# and of either sign: 20 * 20^0.5 * 2^-25 = 3e-6 of a weight; outputs of independent weights are off by as much of
# their size, and the values' own parts (22 bits, cut towards zero) by 2^-22.  Three times that:
GROUP_TOL = 1e-5


def group_errors(out, ref, g):
    """Relative L2 of every (query head, group)."""
    a, b = (np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, g) for x in (out, ref))
    return np.linalg.norm(a - b, axis=-1) / np.linalg.norm(b, axis=-1)


GROUP_SHAPES = [(128, 32, 2, 1), (128, 32, 16, 8), (128, 32, 4, 1), (128, 32, 7, 1), (128, 64, 2, 1), (128, 64, 3, 1), (64, 32, 2, 1),
                (64, 32, 4, 1), (64, 32, 8, 1), (128, 64, 6, 1)]


@pytest.mark.parametrize("d,g,nq,nkv", GROUP_SHAPES)
@pytest.mark.parametrize("S", [1104, 4112])
def test_groups_of_different_scale(torch, d, g, nq, nkv, S):
    """Channel groups of V whose scales lie up to 10^12 apart: every group keeps its own precision."""
    r = np.random.default_rng(d + g + nq + S)
    L = S - 5
    c = Cache(torch, r, 1, nkv, S, d, g, [L])
    q = r.standard_normal((1, nq, d)).astype(np.float32)
    for sizes in ([1, 1e2, 1e3, 1e4], [1e6, 1, 1e-6, 1e2], [1e-12, 1, 1e-4, 1e-8], [0, 1, 1e8, 1e4]):
        x = r.standard_normal((1, nkv, S, d)).astype(np.float32) * np.repeat(np.float32(sizes)[:d // g], g)
        V = set_values(torch, c, x, g)
        out = attend(torch, c.dev, q, [0], [L - 1])
        ref, _ = kv4.attention(q[0], c.val["k"][0, :, :L], V[0, :, :L], 1 / math.sqrt(d))
        zero = np.repeat(np.float32(sizes)[:d // g] == 0, g)
        assert not out[0][:, zero].any()
        err = group_errors(out[0], np.where(zero, 1.0, ref), g)[:, np.float32(sizes)[:d // g] != 0]
        assert (err <= GROUP_TOL).all(), (sizes, err.max(0))


@pytest.mark.parametrize("d,g,nq,nkv", GROUP_SHAPES + [(128, 128, 2, 1), (128, 128, 8, 1), (64, 64, 8, 1)])
@pytest.mark.parametrize("S", [1104, 4112])
@pytest.mark.parametrize("size", [1e6, 1e9])
def test_large_values_of_no_weight(torch, d, g, nq, nkv, S, size):
    """One position whose V is 10^6 or 10^9 times the others' and whose weight is 2^-60 or less, first, in the middle or last in
    the row: nothing of it is seen in the output."""
    r = np.random.default_rng(d + g + nq + S)
    L = S - 5
    q = r.standard_normal((1, nq, d)).astype(np.float32)
    c = Cache(torch, r, 1, nkv, S, d, g, [L])
    kx, vx = ((r.standard_normal((1, nkv, S, d))).astype(np.float32) for _ in range(2))
    for at in (0, 77, L - 1):
        k1, v1 = kx.copy(), vx.copy()
        v1[:, :, at] *= np.float32(size)
        for h in range(nkv):                                  # against all of the KV head's queries
            mine = q[0, h * (nq // nkv):(h + 1) * (nq // nkv)].astype(np.float64)
            away = np.linalg.lstsq(mine, np.full(len(mine), -60.0 * math.sqrt(d)), rcond=None)[0]
            k1[0, h, at] = away
        codes, sb, zb = kv4.quantize(k1, g)
        c.dev.tensors[0].copy_(torch.from_numpy(kv4.pack_rows(codes, True)))
        c.dev.tensors[2].copy_(torch.from_numpy(kv4.pack_words(sb, zb)))
        K, V = kv4.dequantize(codes, sb, zb), set_values(torch, c, v1, g)
        out = attend(torch, c.dev, q, [0], [L - 1])
        ref, m = kv4.attention(q[0], K[0, :, :L], V[0, :, :L], 1 / math.sqrt(d))
        assert m[:, at].max() <= 2.0 ** -58
        assert group_errors(out[0], ref, g).max() <= GROUP_TOL, at


@pytest.mark.parametrize("d,g,nq", [(128, 32, 2), (128, 32, 4), (128, 32, 8), (128, 128, 4), (64, 64, 8), (64, 32, 5)])
@pytest.mark.parametrize("S", [1104, 4112])
def test_large_values_that_one_head_looks_at(torch, d, g, nq, S):
    """A position of large V to which the first query head gives its weight and the others none: either kind of head is right."""
    r = np.random.default_rng(d + g + nq + S + 1)
    L, at = S - 5, 300
    q = r.standard_normal((1, nq, d)).astype(np.float32)
    c = Cache(torch, r, 1, 1, S, d, g, [L])
    kx, vx = ((r.standard_normal((1, 1, S, d))).astype(np.float32) for _ in range(2))
    vx[:, :, at] *= np.float32(1e8)
    goal = np.full(nq, -60.0 * math.sqrt(d))
    goal[0] = 6.0 * math.sqrt(d)
    kx[0, 0, at] = np.linalg.lstsq(q[0].astype(np.float64), goal, rcond=None)[0]
    codes, sb, zb = kv4.quantize(kx, g)
    c.dev.tensors[0].copy_(torch.from_numpy(kv4.pack_rows(codes, True)))
    c.dev.tensors[2].copy_(torch.from_numpy(kv4.pack_words(sb, zb)))
    K, V = kv4.dequantize(codes, sb, zb), set_values(torch, c, vx, g)
    out = attend(torch, c.dev, q, [0], [L - 1])
    ref, m = kv4.attention(q[0], K[0, :, :L], V[0, :, :L], 1 / math.sqrt(d))
    assert np.abs(ref[0]).max() >= 1e5 and np.abs(ref[1:]).max() <= 100
    # the key that answers 6 to one query and -60 to the others is long: its score's terms are some 8 times the others'
    err = group_errors(out[0], ref, g).max(-1)
    assert err[0] <= 8 * GROUP_TOL and err[1:].max() <= GROUP_TOL


@pytest.mark.parametrize("d,g,nq", [(128, 32, 2), (128, 32, 3), (128, 128, 2), (128, 64, 8), (64, 64, 6), (64, 32, 2)])
@pytest.mark.parametrize("S", [1104, 4112])
@pytest.mark.parametrize("rise", [60.0, -60.0, 400.0])
def test_scores_that_rise_while_values_fall(torch, d, g, nq, S, rise):
    """Scores that climb by `rise` octaves along the row while V falls by 10^12 (or the other way round): the positions that
    count are small beside what the row held before."""
    r = np.random.default_rng(d + g + nq + S + 2)
    L = S - 5
    # one dim of each key and query carries the score: a code of 0 or 15 under an exact scale, so that the
    # score itself is rounded three times, 2^-24 * 400 * ln 2 each at most
    ramp = np.linspace(0, rise, S).astype(np.float32)
    kx = np.zeros((1, 1, S, d), np.float32)
    step = kv4.bf16_value(kv4.bf16_bits(np.abs(ramp) / 15)) * 15
    kx[0, 0, :, 3] = np.sign(rise) * step
    q = np.zeros((1, nq, d), np.float32)
    q[0, :, 3] = math.log(2) * math.sqrt(d)
    fall = np.exp2(np.linspace(0, -40, S) * np.sign(rise)).astype(np.float32)
    vx = r.standard_normal((1, 1, S, d)).astype(np.float32) * fall[None, None, :, None]
    c = Cache(torch, r, 1, 1, S, d, g, [L])
    codes, sb, zb = kv4.quantize(kx, g)
    c.dev.tensors[0].copy_(torch.from_numpy(kv4.pack_rows(codes, True)))
    c.dev.tensors[2].copy_(torch.from_numpy(kv4.pack_words(sb, zb)))
    K, V = kv4.dequantize(codes, sb, zb), set_values(torch, c, vx, g)
    out = attend(torch, c.dev, q, [0], [L - 1])
    ref, _ = kv4.attention(q[0], K[0, :, :L], V[0, :, :L], 1 / math.sqrt(d))
    assert group_errors(out[0], ref, g).max() <= GROUP_TOL + 4 * 2.0 ** -24 * abs(rise) * math.log(2)


# ------------------------------------------------------------------ angles
def exact_angles(theta, half):
    """theta^(-i / half) / 2 pi as Decimals of 60 digits, and 2 pi."""
    import decimal
    decimal.getcontext().prec = 60
    two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    ln = decimal.Decimal(float(np.float32(theta))).ln()
    return [(ln * -i / half).exp() / two_pi for i in range(half)], two_pi


@pytest.mark.parametrize("d,theta", [(128, 1e6), (64, 1e6), (128, 1e4), (64, 5e5), (128, 1e12), (64, 3e38), (128, 1.0)])
def test_append_cosines_and_sines(torch, d, theta):
    """Queries whose first half is 1 and whose second half is 0 come out as the cosines and sines: to 0.53 ulp of themselves, plus
    the angle's own error of |position| 2^-65 turns, for any position, the slow pairs' tiny sines among them."""
    half, nq = d // 2, 1
    pos = np.array([0, 1, 2, 3, 17, -1, -5, 100, 4095, 131071, -99999, 2 ** 20 + 1, 999999937, -123456789, 2 ** 31 - 1, -2 ** 31],
                   np.int64)
    T = len(pos)
    qkv = np.zeros((1, T, 3, d), np.float32)
    qkv[0, :, 0, :half] = 1.0
    c = kmr.Kv4Cache.zeros(1, 1, 16, d, 32)
    q = torch.zeros((1, T, nq, d), device="cuda")
    p3 = np.broadcast_to(pos.astype(np.int32), (3, 1, T)).copy()
    kmr.kmr_kv4_append(c, torch.from_numpy(qkv).cuda(), torch.from_numpy(p3).cuda(), i32(torch, [0]), i32(torch, [0]), None, 1, T, nq,
                       None, None, 1e-6, theta, SECTIONS[d], q, None, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    got = q.cpu().numpy()[0, :, 0].astype(np.float64)
    turns, two_pi = exact_angles(theta, half)
    for t, p in enumerate(pos):
        for i in range(half):
            a = turns[i] * int(p)
            a = float((a - a.to_integral_value()) * two_pi)            # within half a turn
            off = abs(int(p)) * 2.0 ** -65 * 2 * math.pi
            for have, want in ((got[t, i], math.cos(a)), (got[t, half + i], math.sin(a))):
                ulp = 0.53 * np.spacing(np.float32(abs(want))) if abs(a) >= 2.0 ** -25 else 2.0 ** -22 * abs(want)
                assert abs(have - want) <= ulp + 1.01 * off, (p, i, have, want)


def test_append_rotations_far_and_near(torch):
    """Random pairs at positions of every size: cosine and sine to 0.53 ulp, two products and their sum, each rounded
    once, of the pair's size."""
    r = np.random.default_rng(91)
    d, nq, T = 128, 2, 64
    pos = (r.choice([-1, 1], (3, 1, T)) * np.floor(2.0 ** r.uniform(0, 31, (3, 1, T)))).astype(np.int64).clip(-2 ** 31, 2 ** 31 - 1)
    qkv = r.standard_normal((1, T, nq + 2, d)).astype(np.float32)
    c = kmr.Kv4Cache.zeros(1, 1, T, d, 32)
    q = torch.zeros((1, T, nq, d), device="cuda")
    kmr.kmr_kv4_append(c, torch.from_numpy(qkv).cuda(), torch.from_numpy(pos.astype(np.int32)).cuda(), i32(torch, [0]), i32(torch, [0]),
                       None, 1, T, nq, None, None, 1e-6, 1e6, SECTIONS[d], q, None, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    got = q.cpu().numpy()[0].astype(np.float64)
    turns, two_pi = exact_angles(1e6, 64)
    for t in range(T):
        for i in range(64):
            axis = 0 if i < 16 else (1 if i < 40 else 2)
            a = turns[i] * int(pos[axis, 0, t])
            a = float((a - a.to_integral_value()) * two_pi)
            x, y = (qkv[0, t, :nq, k].astype(np.float64) for k in (i, i + 64))
            # 0.53 ulp (2^-24 of the value), a product and the sum: 2^-24 each; the angle 2^-34 turns
            tol = (0.53 * 2.0 ** -23 + 2 * 2.0 ** -24 + 2.0 ** -34 * 2 * math.pi) * (np.abs(x) + np.abs(y))
            assert (np.abs(got[t, :, i] - (x * math.cos(a) - y * math.sin(a))) <= tol).all(), (t, i)
            assert (np.abs(got[t, :, i + 64] - (y * math.cos(a) + x * math.sin(a))) <= tol).all(), (t, i)


@pytest.mark.parametrize("d,g,nq,nkv", GROUP_SHAPES + [(128, 128, 2, 1), (64, 64, 8, 1)])
@pytest.mark.parametrize("S", [1104, 4112])
def test_key_groups_of_different_scale(torch, d, g, nq, nkv, S):
    """Channel groups of K up to 10^16 apart, met by queries that are as much smaller there, so that every group has its say
    in the scores: they are off by no more than those of groups alike."""
    r = np.random.default_rng(d + g + nq + S + 3)
    L = S - 5
    c = Cache(torch, r, 1, nkv, S, d, g, [L])
    for sizes in ([1, 1e8, 1e-8, 1e4], [1e-6, 1, 1e6, 1e10], [3e-12, 3e4, 1, 1e-3]):
        size = np.repeat(np.float32(sizes)[:d // g], g)
        codes, sb, zb = kv4.quantize(r.standard_normal((1, nkv, S, d)).astype(np.float32) * size, g)
        c.dev.tensors[0].copy_(torch.from_numpy(kv4.pack_rows(codes, True)))
        c.dev.tensors[2].copy_(torch.from_numpy(kv4.pack_words(sb, zb)))
        q = (r.standard_normal((1, nq, d)).astype(np.float32) / size).astype(np.float32)
        out = attend(torch, c.dev, q, [0], [L - 1])
        ref, _ = kv4.attention(q[0], kv4.dequantize(codes, sb, zb)[0, :, :L], c.val["v"][0, :, :L], 1 / math.sqrt(d))
        assert group_errors(out[0], ref, g).max() <= GROUP_TOL, sizes


@pytest.mark.parametrize("S", [256, 4112])
def test_a_used_slot_filled_anew(torch, S):
    """A slot serves one sequence, then another that is converted into it: with its mass set to 0, as the conversion asks
    for, eviction ranks the new positions by their own weights only; the conversion itself leaves the mass alone."""
    r = np.random.default_rng(S + 7)
    slots, nkv, d, g, nq, L, keep, recent = 3, 2, 64, 32, 4, 200, 40, 5
    cache = kmr.Kv4Cache.zeros(slots, nkv, S, d, g)
    mass = torch.zeros((slots, nkv, S), device="cuda")
    ids, zero, st = i32(torch, [1]), i32(torch, [0]), torch.cuda.current_stream()
    for turn in range(2):
        bits = [kv4.bf16_bits(r.standard_normal((1, nkv, L, d)).astype(np.float32)) for _ in range(2)]
        dev16 = [torch.from_numpy(b.view(np.int16)).cuda() for b in bits]
        if turn:
            left = mass.clone()
            kmr.kmr_kv4_from_bf16(cache, *dev16, 1, L, zero, zero, ids, zero, i32(torch, [L]), 1, L, st)
            assert torch.equal(mass, left) and mass[1, :, :L].min().item() > 0
            mass.index_fill_(0, ids.long(), 0.0)
        else:
            kmr.kmr_kv4_from_bf16(cache, *dev16, 1, L, zero, zero, ids, zero, i32(torch, [L]), 1, L, st)
        vals = [kv4.dequantize(*kv4.quantize(kv4.bf16_value(b[0]), g)) for b in bits]
        total = np.zeros((nkv, L))
        for _ in range(3):
            q = r.standard_normal((1, nq, d)).astype(np.float32) * 2
            attend(torch, cache, q, [1], [L - 1], mass)
            total += kv4.attention(q[0], vals[0], vals[1], 1 / math.sqrt(d))[1]
        assert kmr.kmr_last_device_error() == 0
        got = mass[1, :, :L].cpu().numpy()
        assert np.allclose(got, total, rtol=4 * ATTN_TOL, atol=1e-30)
        dst = kmr.Kv4Cache.zeros(1, nkv, 48, d, g)
        kept, new = evict(torch, cache, dst, [1], [0], [L], keep, recent, mass, None)
        assert kmr.kmr_last_device_error() == 0
        for h in range(nkv):
            assert kept[0, h].tolist() == kv4.evict_positions(got[h], L, keep, recent)


def test_evict_refused_rows_stand_in_no_way(torch):
    """Rows refused for their own slots or length name a good row's destination and, as sources, another's: both move."""
    r = np.random.default_rng(95)
    slots, nkv, S, d, g, keep = 8, 2, 64, 64, 32, 10
    c = Cache(torch, r, slots, nkv, S, d, g)
    before = c.host()
    m = r.random((slots, nkv, S)).astype(np.float32)
    big = 2 ** 31 - 1
    #      good  good   length  length  slot     slot    source of a refused row is a good row's destination
    ids, dids, n = [0, 1, 2, 3, 8, -1, 7, 6], [7, 6, 7, 6, 7, 6, 2, big], [40, 5, 65, -1, 20, 20, 65, 20]
    kept, new = evict(torch, c.dev, c.dev, ids, dids, n, keep, 3, torch.from_numpy(m.copy()).cuda(), None)
    assert kmr.kmr_last_device_error() in (kmr.KMR_ERR_SLOT_RANGE, kmr.KMR_ERR_CACHE_FULL)
    assert new.tolist() == [keep, 5, 0, 0, 0, 0, 0, 0] and (kept[2:] == -1).all()
    got = c.host()
    for a, w in zip(got, before):
        assert np.array_equal(a[:6], w[:6])
        for src, dst, k, b in ((0, 7, keep, 0), (1, 6, 5, 1)):
            for h in range(nkv):
                want = kv4.evict_positions(m[src, h], n[b], keep, 3)
                assert kept[b, h, :k].tolist() == want
                assert np.array_equal(a[dst, h, :k], w[src, h, want]) and np.array_equal(a[dst, h, k:], w[dst, h, k:])


@pytest.mark.parametrize("d,g,nq", [(128, 32, 2), (128, 32, 4), (128, 32, 8), (128, 64, 1), (128, 128, 6), (64, 64, 8), (64, 32, 3)])
@pytest.mark.parametrize("S", [512, 1104, 4112])
def test_scores_that_step_up_beside_large_values_of_no_weight(torch, d, g, nq, S):
    """Two steps of 40 octaves in the scores where V falls by 2^30, and in every 16 positions one of no weight whose V is 2^40: what
    counts is small beside what the row held before and beside what it holds now."""
    r = np.random.default_rng(d + g + nq + S + 4)
    L = S - 5
    octaves = np.floor(np.arange(S) * 3 / S) * 40.0
    out_of = np.arange(S) % 16 == 5
    octaves[out_of] = -120.0
    # one dim carries the score, as a code of 0 or 15 under an exact scale
    kx = np.zeros((1, 1, S, d), np.float32)
    kx[0, 0, :, 3] = np.sign(octaves) * kv4.bf16_value(kv4.bf16_bits((np.abs(octaves) / 15).astype(np.float32))) * 15
    q = np.zeros((1, nq, d), np.float32)
    q[0, :, 3] = math.log(2) * math.sqrt(d)
    vx = r.standard_normal((1, 1, S, d)).astype(np.float32)
    vx[0, 0] *= np.exp2(np.where(out_of, 40, -30 * np.floor(np.arange(S) * 3 / S))).astype(np.float32)[:, None]
    c = Cache(torch, r, 1, 1, S, d, g, [L])
    codes, sb, zb = kv4.quantize(kx, g)
    c.dev.tensors[0].copy_(torch.from_numpy(kv4.pack_rows(codes, True)))
    c.dev.tensors[2].copy_(torch.from_numpy(kv4.pack_words(sb, zb)))
    K, V = kv4.dequantize(codes, sb, zb), set_values(torch, c, vx, g)
    out = attend(torch, c.dev, q, [0], [L - 1])
    ref, _ = kv4.attention(q[0], K[0, :, :L], V[0, :, :L], 1 / math.sqrt(d))
    # scores of 80 octaves, rounded three times; outputs of positions that count alike
    assert group_errors(out[0], ref, g).max() <= GROUP_TOL + 4 * 2.0 ** -24 * 80 * math.log(2)


@pytest.mark.parametrize("seed", range(40))
def test_attention_of_wild_scales(torch, seed):
    """Random shapes; V scales that differ by up to 2^60 between positions, groups or both, rows and groups of zeros or
    constants among them; scores of up to 100 octaves."""
    r = np.random.default_rng(seed + 1000)
    d = int(r.choice([64, 128]))
    g = int(r.choice([x for x in (32, 64, 128) if x <= d]))
    nkv, rep, S = int(r.choice([1, 2])), int(r.integers(1, 9)), int(r.choice([64, 208, 512, 1104, 2064, 4112]))
    L, ng, nq = int(r.integers(S // 2, S + 1)), d // g, nkv * rep
    c = Cache(torch, r, 1, nkv, S, d, g, [L])
    e = np.zeros((1, nkv, S, ng))
    if seed % 4 in (1, 3):
        e = e + r.uniform(-30, 30, (1, 1, 1, ng))
    if seed % 4 in (2, 3):
        e = e + r.uniform(-30, 30, (1, nkv, S, 1 if seed % 8 < 4 else ng))
    x = (r.standard_normal((1, nkv, S, d)) * np.exp2(np.repeat(e, g, -1))).astype(np.float32)
    if seed % 3 == 0:
        x[r.random((1, nkv, S)) < 0.5] = 0
    if seed % 5 == 0:
        x = np.where(np.repeat(r.random((1, nkv, S, ng)) < 0.3, g, -1), np.float32(1.5), x)
    V = set_values(torch, c, x, g)[0, :, :L]
    q = (r.standard_normal((1, nq, d)) * r.choice([0.1, 1, 3, 10])).astype(np.float32)
    out = attend(torch, c.dev, q, [0], [L - 1])[0]
    K = c.val["k"][0, :, :L]
    ref, _ = kv4.attention(q[0], K, V, 1 / math.sqrt(d))
    assert np.isfinite(out).all()
    for i in range(nq):
        h = i // rep
        # a score is a sum of codes (not centred: up to 15 s beside the base, so twice the group's largest |k|) times the query,
        # off by some 3 * 2^-22 of the terms' size; a weight by as much of itself; the values' parts and sums by 3e-6
        big = np.abs(K[h]).reshape(L, ng, g).max(-1).repeat(g, -1) * 2
        off = 3e-6 + 3 * 2.0 ** -22 * (big @ np.abs(q[0, i].astype(np.float64))).max() / math.sqrt(d) / math.log(2)
        a = K[h] @ q[0, i].astype(np.float64) / math.sqrt(d)
        p = np.exp(a - a.max())
        size = (p / p.sum()) @ np.abs(V[h]).reshape(L, ng, g).max(-1)
        assert (np.abs(out[i] - ref[i]) <= off * np.repeat(size, g) + 1e-37).all(), (i, d, g, rep, S, L)


@pytest.mark.parametrize("d", [64, 128])
def test_appended_queries_and_keys_round_as_a_plain_norm_and_rotation(torch, d):
    """Next to the same operations one by one in single precision (squares, their mean, reciprocal root, products, cosine and
    sine of 64-bit angles rounded once, products, sums): the bits agree but where a cosine or sine lies within 0.03 steps of
    a border, so that the codes, which a last bit can move by one, are the same ones."""
    r = np.random.default_rng(d + 5)
    B, T, nq, nkv, g = 2, 300, 8, 4, 32
    gen = torch.Generator(device="cuda").manual_seed(d)
    qkv = torch.randn((B, T, nq + 2 * nkv, d), generator=gen, device="cuda") * 2
    pos = i32(torch, r.integers(-100, 20000, (3, B, T)))
    w = [(1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).bfloat16() for _ in range(2)]
    q = torch.zeros((B, T, nq, d), device="cuda")
    c = kmr.Kv4Cache.zeros(B, nkv, 304, d, g)
    kmr.kmr_kv4_append(c, qkv, pos, i32(torch, [0, 1]), i32(torch, [0, 0]), None, B, T, nq, w[0], w[1], 1e-6, 1e6, SECTIONS[d], q, None,
                       torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    f = torch.arange(d // 2, device="cuda")
    a, b, _ = SECTIONS[d]
    ang = pos.double()[(f >= a).long() + (f >= a + b).long()].permute(1, 2, 0) * torch.pow(
        torch.tensor(1e6, dtype=torch.float64, device="cuda"), -2.0 * f.double() / d)
    cs, sn = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    plain = []
    for x, wt in ((qkv[:, :, :nq], w[0]), (qkv[:, :, nq:nq + nkv], w[1])):
        # the mean's order: 32 dims apart, then neighbours
        s = x.square().unflatten(-1, (d // 32, 32))
        total = s[..., 0, :]
        for k in range(1, d // 32):
            total = total + s[..., k, :]
        while total.shape[-1] > 1:
            total = total[..., 0::2] + total[..., 1::2]
        y = x * torch.rsqrt(total * (1.0 / d) + 1e-6) * wt.float()
        lo, hi = y[..., :d // 2], y[..., d // 2:]
        plain.append(torch.cat((lo * cs - hi * sn, hi * cs + lo * sn), -1))
    # on average an error of 0.001 steps either side of a border, of a cosine or a sine, which each value takes both of
    assert (q != plain[0]).float().mean().item() <= 0.005
    codes, sb, zb = kv4.quantize(plain[1].transpose(1, 2).cpu().numpy(), g)
    got = c.host() if hasattr(c, "host") else [t.cpu().numpy() for t in c.tensors]
    assert (kv4.unpack_rows(got[0][:, :, :T], True) != codes).mean() <= 2e-5
