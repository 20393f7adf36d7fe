"""GPU parity of the router, the int4 experts and the adapters against their oracle, and a run of them together."""
import numpy as np
import pytest

from gpu_helpers import rel_l2, require_gpu
import int4_weight_only_group_gb300 as kmr
from oracle import moe

pytestmark = pytest.mark.gpu

# A row's result against 64 bits, relative L2.  fp32: operands hold 22 bits or more of their row's largest value, and a
# tensor-core sum of K products in steps of 16 loses up to an ulp (2^-23) of the running sum at each: for the longest
# rows here (8192 + 8192 remainders: 1024 steps, of which half an ulp on average and 0.6 of the final size) 4e-5, over the
# three products of an expert.  bf16: half a step of the result, 2^-8 of it at most, and half a step of fp16, 2^-11, for the
# activations between the products, which the down product's sum hands on at about its own size.
TOL = {kmr.KMR_F32: 4e-5, kmr.KMR_BF16: 2.0 ** -8 + 2.0 ** -10}
DT = [kmr.KMR_F32, kmr.KMR_BF16]


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


def tdt(torch, dtype):
    return torch.bfloat16 if dtype == kmr.KMR_BF16 else torch.float32


def i32(torch, a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def rounded(torch, a, dtype):
    """a as the device holds it, and its values."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(tdt(torch, dtype))
    return t, t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ router
def route(torch, logits, k, renorm, dtype, stream=None):
    T, E = logits.shape
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    kmr.kmr_moe_route(logits, dtype, T, E, k, renorm, ids, w, stream or torch.cuda.current_stream())
    return ids, w


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (5, 33, 32), (517, 60, 4), (64, 7, 7), (130, 1024, 10), (9, 256, 1), (3, 1000, 32)])
def test_route(torch, T, E, k, dtype):
    r = np.random.default_rng(T * 1000 + E)
    a = r.standard_normal((T, E)) * 2
    a[r.random((T, E)) < 0.2] = -np.inf
    a[r.random((T, E)) < 0.02] = np.nan
    a = np.round(a * 8) / 8 if T > 100 else a                 # many ties
    a[T // 2] = -np.inf
    if T > 8:
        a[0] = 0.0
        a[1, : E // 2] = -0.0
        a[2, E - 1] = np.inf
        a[3, 0] = a[3, E // 2] = np.inf
        a[4] = np.nan
        a[5] = -3e38
    dev, val = rounded(torch, a, dtype)
    for renorm in (False, True):
        ids, w = route(torch, dev, k, renorm, dtype)
        want_ids, want = moe.route(val, k, renorm)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        # exp to 2 ulp, its argument and the quotient half an ulp each (the argument up to 16 in size: 16 ulp of 1), the sum
        # of E positive terms over lanes 5 + E / 32 roundings
        assert np.allclose(w.cpu().numpy(), want, rtol=(24 + E / 32) * 2.0 ** -24, atol=1e-38)
    assert kmr.kmr_last_device_error() == 0


# ------------------------------------------------------------------ experts
class Layer:
    def __init__(self, torch, r, E, H, I, scale=1.0):
        self.shape = (E, H, I)
        self.gate_up, self.down, packed = [], [], []
        for N, K, flags, keep in ((2 * I, H, kmr.KMR_PACK_GATE_UP, self.gate_up), (H, I, 0, self.down)):
            size = kmr.kmr_packed_size(N, K)
            out = torch.empty((E, size), dtype=torch.uint8, device="cuda")
            for e in range(E):
                q = r.integers(0, 16, (N, K), dtype=np.uint8)
                s = torch.from_numpy((r.uniform(0.002, 0.02, (N, K // 128)) * scale).astype(np.float32)).bfloat16()
                z = torch.from_numpy((r.standard_normal((N, K // 128)) * 0.005 * scale).astype(np.float32)).bfloat16()
                keep.append(moe.dense(q, s.float().numpy(), z.float().numpy()))
                kmr.kmr_pack_int4(torch.from_numpy(q).cuda(), s.cuda(), z.cuda(), N, K, 128, flags, out[e], size, True,
                                  torch.cuda.current_stream())
            packed.append(out)
        self.dev = kmr.Moe(*packed, E, H, I, 128, torch.cuda.current_stream())


def run_experts(torch, layer, x, ids, w, dtype, y=None, epilogue=kmr.KMR_EPI_NONE, stream=None):
    T, k = ids.shape
    n = kmr.kmr_moe_experts_workspace_size(layer.dev, dtype, T, k)
    assert n > 0
    ws = torch.full(((n + 3) // 4,), float("nan"), device="cuda")
    if y is None:
        y = torch.full((T, layer.shape[1]), float("nan"), device="cuda", dtype=tdt(torch, dtype))
    kmr.kmr_moe_experts(layer.dev, x, dtype, ids, w, T, k, y, epilogue, ws, n, stream or torch.cuda.current_stream())
    return y


def places(r, T, E, k, none=0.1):
    ids = np.stack([r.permutation(max(E, k))[:k] for _ in range(T)]) % E
    ids[r.random((T, k)) < none] = -1
    w = r.random((T, k)).astype(np.float32)
    w[ids < 0] = np.nan                                       # not read
    return ids.astype(np.int32), w


def rows_close(got, want, tol):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    for t in range(len(want)):
        assert rel_l2(got[t], want[t]) <= tol, (t, rel_l2(got[t], want[t]))


SHAPES = [  # E, H, I, T, k
    (8, 256, 128, 1, 2), (1, 128, 128, 3, 1), (16, 512, 384, 33, 4), (5, 384, 256, 7, 8), (4, 2048, 768, 2, 3), (60, 256, 128, 100, 4),
    (2, 2176, 128, 5, 2), (2, 256, 2176, 5, 2), (1, 8192, 128, 2, 1), (1, 128, 8192, 2, 1), (2, 4096, 4096, 1, 2), (3, 640, 1408, 40, 2),
    (8, 512, 256, 300, 2), (2, 256, 384, 257, 1), (2, 8192, 128, 40, 1), (2, 128, 8192, 40, 1), (3, 256, 2176, 700, 2),
    (40, 256, 128, 1200, 8), (200, 128, 128, 64, 6), (4, 2048, 768, 90, 2), (1, 128, 128, 2081, 32),
    # few tokens whose tiles pass through the rings more than once, the most tokens and places of that form and one more of
    # each; more places than one pass takes
    (6, 4096, 1024, 4, 3), (12, 1024, 4096, 4, 3), (7, 640, 2560, 16, 2), (7, 640, 2560, 17, 1), (7, 640, 2560, 11, 3),
    (2, 8192, 1024, 3, 2), (4, 128, 256, 17000, 2),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("E,H,I,T,k", SHAPES)
def test_experts(torch, E, H, I, T, k, dtype):
    r = np.random.default_rng(E * H + I + T)
    layer = Layer(torch, r, E, H, I)
    x, xv = rounded(torch, r.standard_normal((T, H)) * np.exp(r.standard_normal((T, 1))), dtype)
    ids, w = places(r, T, E, k)
    if T > 2:
        ids[1] = -1                                           # a padded token
        ids[2] = ids[2, 0] if ids[2, 0] >= 0 else 0           # one expert in every place
        w[2] = 0.25
    kmr.kmr_smem_poison(0x7FC07FC0, torch.cuda.current_stream())
    dev_ids, dev_w = i32(torch, ids), torch.from_numpy(w).cuda()
    y = run_experts(torch, layer, x, dev_ids, dev_w, dtype)
    assert kmr.kmr_last_device_error() == 0
    want = moe.experts(xv, ids, w, layer.gate_up, layer.down)
    rows_close(y, want, TOL[dtype])
    # added to what is there, in place over x
    z = x.clone()
    run_experts(torch, layer, z, dev_ids, dev_w, dtype, z, kmr.KMR_EPI_RESIDUAL)
    rows_close(z, want + xv, TOL[dtype])
    assert kmr.kmr_last_device_error() == 0
    again = run_experts(torch, layer, x, dev_ids, dev_w, dtype)
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [1, 4, 40, 300])
def test_all_tokens_to_one_expert(torch, T, dtype):
    r = np.random.default_rng(T)
    layer = Layer(torch, r, 9, 256, 256)
    x, xv = rounded(torch, r.standard_normal((T, 256)), dtype)
    ids, w = np.full((T, 1), 7, np.int32), r.random((T, 1)).astype(np.float32)
    y = run_experts(torch, layer, x, i32(torch, ids), torch.from_numpy(w).cuda(), dtype)
    rows_close(y, moe.experts(xv, ids, w, layer.gate_up, layer.down), TOL[dtype])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [3, 50])
def test_experts_bad_ids_and_values(torch, T, dtype):
    """Ids out of range are places without an expert and are reported; NaN and infinities stay in their token."""
    r = np.random.default_rng(11)
    E, H, I, k = 6, 256, 128, 3
    layer = Layer(torch, r, E, H, I)
    x, xv = rounded(torch, r.standard_normal((T, H)), dtype)
    x[0, 5] = float("nan")
    x[1, 7] = float("inf")
    ids, w = places(r, T, E, k)
    ids[0, 0] = ids[1, 0] = 2
    ids[2] = [E, 2, -2]
    w[2] = [np.nan, 0.5, np.inf]
    y = run_experts(torch, layer, x, i32(torch, ids), torch.from_numpy(w).cuda(), dtype)
    assert kmr.kmr_last_device_error() == kmr.KMR_ERR_INVALID_ARG
    got = y.float().cpu().numpy()
    assert not np.isfinite(got[:2]).any()
    rows_close(y[2:], moe.experts(xv, ids, w, layer.gate_up, layer.down)[2:], TOL[dtype])
    ids[:] = -1                                               # nothing at all
    y = run_experts(torch, layer, x, i32(torch, ids), torch.from_numpy(w).cuda(), dtype)
    assert kmr.kmr_last_device_error() == 0 and (y == 0).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,x_size,w_size", [(2, 1e-30, 1.0), (2, 1e15, 1e-6), (70, 1e-30, 1.0), (70, 1e15, 1e-6), (70, 1.0, 2.0 ** -60),
                                             (70, 1e-4, 2.0 ** 20), (2, 1.0, 2.0 ** -60)])
def test_experts_far_scales(torch, T, x_size, w_size, dtype):
    """Inputs and weights far from one keep their precision (the 64-bit sums show no overflow in single precision)."""
    r = np.random.default_rng(5)
    layer = Layer(torch, r, 4, 256, 256, w_size)
    x, xv = rounded(torch, r.standard_normal((T, 256)) * x_size, dtype)
    ids, w = places(r, T, 4, 2, 0.0)
    want = moe.experts(xv, ids, w, layer.gate_up, layer.down)
    assert 1e-36 < np.abs(want).max() < 1e38 or np.abs(want).max() < 1e-36
    y = run_experts(torch, layer, x, i32(torch, ids), torch.from_numpy(w).cuda(), dtype)
    if np.abs(want).max() > 1e-30:
        rows_close(y, want, TOL[dtype])
    else:
        assert np.abs(y.double().cpu().numpy()).max() <= 1e-28


@pytest.mark.parametrize("dtype", DT)
def test_a_token_by_itself(torch, dtype):
    """A token's bits do not depend on the other tokens of a call of the same form."""
    r = np.random.default_rng(8)
    layer = Layer(torch, r, 8, 512, 384)
    x, _ = rounded(torch, r.standard_normal((9, 512)), dtype)
    ids, w = places(r, 9, 8, 3, 0.0)
    ids, w = i32(torch, ids), torch.from_numpy(w).cuda()
    few = run_experts(torch, layer, x[:4], ids[:4], w[:4], dtype)
    for t in range(4):
        assert torch.equal(run_experts(torch, layer, x[t:t + 1], ids[t:t + 1], w[t:t + 1], dtype)[0], few[t])


@pytest.mark.parametrize("dtype", DT)
def test_tokens_among_others_when_grouped(torch, dtype):
    """The same for the grouped form, whose tiles hold other tokens and numbers of tokens in either call."""
    r = np.random.default_rng(9)
    layer = Layer(torch, r, 8, 512, 384)
    x, _ = rounded(torch, r.standard_normal((700, 512)), dtype)
    ids, w = places(r, 700, 8, 3, 0.0)
    ids, w = i32(torch, ids), torch.from_numpy(w).cuda()
    many = run_experts(torch, layer, x, ids, w, dtype)
    for a, b in ((0, 12), (30, 130), (300, 650)):
        assert torch.equal(run_experts(torch, layer, x[a:b], ids[a:b], w[a:b], dtype), many[a:b])


def test_experts_in_a_larger_workspace(torch):
    """A workspace for many tokens serves any number of them, whatever an earlier call has left in it."""
    r = np.random.default_rng(22)
    layer = Layer(torch, r, 6, 256, 2176)
    n = kmr.kmr_moe_experts_workspace_size(layer.dev, kmr.KMR_BF16, 60, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream()
    for T in (60, 16, 1, 17, 59, 3):
        x, xv = rounded(torch, r.standard_normal((T, 256)), kmr.KMR_BF16)
        ids, w = places(r, T, 6, 2)
        y = torch.full((T, 256), float("nan"), device="cuda", dtype=torch.bfloat16)
        kmr.kmr_moe_experts(layer.dev, x, kmr.KMR_BF16, i32(torch, ids), torch.from_numpy(w).cuda(), T, 2, y, kmr.KMR_EPI_NONE, ws, n, stream)
        rows_close(y, moe.experts(xv, ids, w, layer.gate_up, layer.down), TOL[kmr.KMR_BF16])
    assert kmr.kmr_last_device_error() == 0


def test_experts_captured_and_on_two_streams(torch):
    r = np.random.default_rng(21)
    layer = Layer(torch, r, 16, 512, 256)
    cases = []
    for T, dtype in ((2, kmr.KMR_F32), (200, kmr.KMR_BF16)):
        x, _ = rounded(torch, r.standard_normal((T, 512)), dtype)
        ids, w = places(r, T, 16, 4)
        ids, w = i32(torch, ids), torch.from_numpy(w).cuda()
        n = kmr.kmr_moe_experts_workspace_size(layer.dev, dtype, T, 4)
        cases.append((x, ids, w, dtype, torch.empty(n, dtype=torch.uint8, device="cuda"), n, run_experts(torch, layer, x, ids, w, dtype)))

    def go(c, y, stream):
        kmr.kmr_moe_experts(layer.dev, c[0], c[3], c[1], c[2], c[1].shape[0], 4, y, kmr.KMR_EPI_NONE, c[4], c[5], stream)

    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s, c in zip(streams, cases):
        outs.append([torch.zeros_like(c[6]) for _ in range(8)])
    torch.cuda.synchronize()
    for i in range(8):
        for s, c, o in zip(streams, cases, outs):
            go(c, o[i], s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        for y in o:
            assert torch.equal(y, c[6])
    for c in cases:                                          # captured, with other values at replay
        y = torch.zeros_like(c[6])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(c, y, torch.cuda.current_stream())
        for scale in (1.0, -0.5):
            c[0].mul_(scale)
            c[1].copy_(torch.flip(c[1], (0,)))
            want = run_experts(torch, layer, c[0], c[1], c[2], c[3])
            g.replay()
            torch.cuda.synchronize()
            # bit for bit: places that were without an expert have a weight of NaN
            bits = torch.int16 if y.dtype == torch.bfloat16 else torch.int32
            assert torch.equal(y.view(bits), want.view(bits))
    assert kmr.kmr_last_device_error() == 0


# ------------------------------------------------------------------ adapters
def adapter_set(torch, r, L, K, N, rank, ranks=None):
    a = torch.from_numpy((r.standard_normal((L, rank, K)) * K ** -0.5).astype(np.float32)).bfloat16().cuda()
    b = torch.from_numpy((r.standard_normal((L, N, rank)) * 0.3).astype(np.float32)).bfloat16().cuda()
    scales = torch.from_numpy(r.uniform(0.25, 2, L).astype(np.float32)).cuda()
    host = [t.float().cpu().numpy() for t in (a, b)] + [ranks if ranks is not None else np.full(L, rank), scales.cpu().numpy()]
    if ranks is not None:
        for i, n in enumerate(ranks):                        # past an adapter's rank: anything
            a[i, max(n, 0):] = float("nan")
            b[i, :, max(n, 0):] = float("inf")
    return kmr.Lora(a, b, None if ranks is None else i32(torch, ranks), scales), host


# v and y are sums of K and r products whose factors are exact (three terms of 8 bits), in fp32: K / 16 + r / 16 steps of half an
# ulp at 0.6 of the size, three terms each, 6144 + 128: 4e-5.  bf16 results: half a step.
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,K,N,rank,L", [(1, 128, 64, 8, 2), (3, 2048, 512, 16, 8), (16, 256, 4096, 64, 32), (64, 160, 48, 24, 3),
                                          (65, 512, 16, 128, 5), (77, 16, 272, 40, 4), (500, 256, 128, 16, 7), (2049, 128, 96, 32, 6),
                                          (2300, 192, 144, 128, 3), (40, 6144, 32, 8, 2), (1, 16, 16, 8, 1), (305, 80, 144, 128, 5),
                                          (1300, 1040, 272, 64, 9), (5000, 48, 16, 32, 700), (304, 2048, 1040, 56, 300)])
def test_lora(torch, T, K, N, rank, L, dtype):
    r = np.random.default_rng(T + K)
    lora, host = adapter_set(torch, r, L, K, N, rank)
    x, xv = rounded(torch, r.standard_normal((T, K)) * np.exp(2 * r.standard_normal((T, 1))), dtype)
    base, bv = rounded(torch, r.standard_normal((T, N)), dtype)
    runs = np.repeat(r.integers(-1, L, T), r.integers(1, 40, T))[:T] if T > 70 else r.integers(-1, L, T)
    ids = i32(torch, runs)
    want = moe.adapters(xv, bv, runs, *host)
    delta = moe.adapters(xv, np.zeros_like(bv), runs, *host)
    stream = torch.cuda.current_stream()
    kmr.kmr_smem_poison(0x7FC07FC0, stream)
    y = torch.full((T, N), float("nan"), device="cuda", dtype=x.dtype)
    kmr.kmr_lora_apply(lora, x, base, y, dtype, ids, T, K, N, stream)
    rows_close(y, want, TOL[dtype])
    y.fill_(float("nan"))
    kmr.kmr_lora_apply(lora, x, None, y, dtype, ids, T, K, N, stream)
    assert torch.equal(y[ids < 0], torch.zeros_like(y[ids < 0]))
    rows_close(y, delta, TOL[dtype])
    # in place, on some columns of wider rows, x among other columns too
    wide = torch.full((T, N + 32), 7.0, device="cuda", dtype=x.dtype)
    wide[:, 16:16 + N] = base
    wx = torch.full((T, K + 8), float("nan"), device="cuda", dtype=x.dtype)
    wx[:, 8:] = x
    part = wide[:, 16:16 + N]
    kmr.kmr_lora_apply(lora, wx[:, 8:], part, part, dtype, ids, T, K + 8, N + 32, stream)
    rows_close(part, want, TOL[dtype])
    assert torch.equal(part[ids < 0], base[ids < 0])
    assert (wide[:, :16] == 7).all() and (wide[:, 16 + N:] == 7).all()
    assert kmr.kmr_last_device_error() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [7, 90, 2100])
def test_lora_ranks_bad_ids_and_values(torch, T, dtype):
    r = np.random.default_rng(T)
    K, N, L = 256, 96, 5
    ranks = np.array([16, 0, 5, 40, 33])
    lora, host = adapter_set(torch, r, L, K, N, 40, ranks)
    x, xv = rounded(torch, r.standard_normal((T, K)), dtype)
    base, bv = rounded(torch, r.standard_normal((T, N)), dtype)
    runs = r.integers(0, L, T)
    runs[3], runs[4], runs[5] = L, -2, 3
    x[5, 9] = float("nan")
    ids = i32(torch, runs)
    y = torch.zeros((T, N), device="cuda", dtype=x.dtype)
    kmr.kmr_lora_apply(lora, x, base, y, dtype, ids, T, K, N, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == kmr.KMR_ERR_INVALID_ARG
    want = moe.adapters(xv, bv, runs, *host)
    assert torch.isnan(y[5]).all() and torch.equal(y[3:5], base[3:5])
    keep = [t for t in range(T) if t != 5]
    rows_close(y[keep], want[keep], TOL[dtype])


@pytest.mark.parametrize("dtype", DT)
def test_lora_captured_and_on_two_streams(torch, dtype):
    r = np.random.default_rng(31)
    K, N, L = 320, 208, 9
    lora, _ = adapter_set(torch, r, L, K, N, 16)
    cases = []
    for T in (5, 900):
        x, _ = rounded(torch, r.standard_normal((T, K)), dtype)
        base, _ = rounded(torch, r.standard_normal((T, N)), dtype)
        ids, want = i32(torch, r.integers(-1, L, T)), torch.empty_like(base)
        kmr.kmr_lora_apply(lora, x, base, want, dtype, ids, T, K, N, torch.cuda.current_stream())
        cases.append((x, base, ids, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.zeros_like(c[3]) for _ in range(8)] for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for s, c, o in zip(streams, cases, outs):
            kmr.kmr_lora_apply(lora, c[0], c[1], o[i], dtype, c[2], len(c[2]), K, N, s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, c[3]) for c, o in zip(cases, outs) for y in o)
    for x, base, ids, want in cases:                         # captured, with other values at replay
        y = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kmr.kmr_lora_apply(lora, x, base, y, dtype, ids, len(ids), K, N, torch.cuda.current_stream())
        for scale in (1.0, -0.5):
            x.mul_(scale)
            ids.copy_(torch.flip(ids, (0,)))
            kmr.kmr_lora_apply(lora, x, base, want, dtype, ids, len(ids), K, N, torch.cuda.current_stream())
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
    assert kmr.kmr_last_device_error() == 0


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T,dtype", [(1, kmr.KMR_F32), (6, kmr.KMR_F32), (90, kmr.KMR_BF16), (200, kmr.KMR_F32)])
def test_layer_of_adapters_router_and_experts(torch, T, dtype):
    """A layer's second half as a user runs it: the O projection (the int4 GEMV for a few rows) with each request's
    adapter, then the router and the experts added to the residual."""
    r = np.random.default_rng(T + 3)
    H, I, E, k, L = 256, 128, 12, 3, 4
    layer = Layer(torch, r, E, H, I)
    lora, host = adapter_set(torch, r, L, H, H, 16)
    stream = torch.cuda.current_stream()
    x, xv = rounded(torch, r.standard_normal((T, H)), dtype)
    Wr = r.standard_normal((E, H)) * 0.1
    runs = r.integers(-1, L, T)
    if T <= 16 and dtype == kmr.KMR_F32:
        q = r.integers(0, 16, (H, H), dtype=np.uint8)
        s, z = (torch.from_numpy((r.uniform(0.002, 0.02, (H, H // 128))).astype(np.float32)).bfloat16() for _ in range(2))
        size = kmr.kmr_packed_size(H, H)
        packed = torch.empty(size, dtype=torch.uint8, device="cuda")
        kmr.kmr_pack_int4(torch.from_numpy(q).cuda(), s.cuda(), z.cuda(), H, H, 128, 0, packed, size, True, stream)
        base = torch.zeros((T, H), device="cuda")
        kmr.kmr_int4_gemv(packed, H, H, 128, 0, x, T, base, kmr.KMR_EPI_NONE, stream)
        bv = base.double().cpu().numpy()
        assert rel_l2(bv, xv @ moe.dense(q, s.float().numpy(), z.float().numpy()).T) <= 1e-2
    else:
        base, bv = rounded(torch, r.standard_normal((T, H)), dtype)
    h = base.clone()
    kmr.kmr_lora_apply(lora, x, h, h, dtype, i32(torch, runs), T, H, H, stream)
    hv = h.double().cpu().numpy()
    rows_close(h, moe.adapters(xv, bv, runs, *host), TOL[dtype])
    logits, lv = rounded(torch, hv @ Wr.T, kmr.KMR_F32)
    ids, w = route(torch, logits, k, True, kmr.KMR_F32)
    want_ids, want_w = moe.route(lv, k, True)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    y = h.clone()
    run_experts(torch, layer, h, ids, w, dtype, y, kmr.KMR_EPI_RESIDUAL)
    rows_close(y, hv + moe.experts(hv, want_ids, want_w, layer.gate_up, layer.down), TOL[dtype])
    assert kmr.kmr_last_device_error() == 0
