"""GPU parity of the int4 experts where weight rows, scales and inputs differ in size, and the adapters' last bits."""
import numpy as np
import pytest

from gpu_helpers import rel_l2, require_gpu
from test_gpu_moe import SHAPES
import int4_weight_only_group_gb300 as kmr
from oracle import moe

pytestmark = pytest.mark.gpu
DT = [kmr.KMR_F32, kmr.KMR_BF16]

# A row's result against 64 bits, relative L2.
# fp32: each of the three products takes, for every group of 128 inputs, at most 9 full-size steps of the tensor cores (8 of the
# codes, one of the zero points), which cut the running sum off at some 2^-25 of it each, always towards zero: 9 x 2^-25 = 2.7e-7.  The
# inputs of both products are held in two fp16 terms (half a step: 2^-23 at the most, 0.7e-7 rms), the groups' sums are
# added in fp32 (up to 64 additions of 2^-24, at random: 2.8e-7 rms at their final size, 0.6 of it on the way) and silu takes
# 4 roundings.  The gate's error counts up to 1.3 times (silu's slope against its value, for gates of size 1): 2.7 x (1.3 + 1 +
# 1) + (2.8 + 0.7) x sqrt(3) = 1.5e-6, and 2e-6 with silu and the weighted sum's roundings.
# bf16: the result's rounding is half a step at the most, uniform: 2^-8 / sqrt(3) rms where all values stand at the lower end
# of their binade, 2.26e-3, and 4 deviations of its own for 128 columns 16% more.  The activations and, of many tokens, each expert's
# result are held as fp16: half a step, 2^-11, each.  2.62e-3 + 2 x 4.9e-4.
TOL = {kmr.KMR_F32: 2e-6, kmr.KMR_BF16: 3.6e-3}


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


def rounded(torch, a, dtype):
    """a as the device holds it, and its values."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16 if dtype == kmr.KMR_BF16 else torch.float32)
    return t, t.float().cpu().numpy().astype(np.float64)


class Layer:
    """Experts whose scales and zeros are given: s and z [E][N, K / 128] of gate_up and of down; inputs `eights` have codes of 8."""

    def __init__(self, torch, r, H, I, gate_up, down, eights=()):
        E = len(gate_up[0])
        self.shape, self.gate_up, self.down, packed = (E, H, I), [], [], []
        for (ss, zz), N, K, flags, keep in ((gate_up, 2 * I, H, kmr.KMR_PACK_GATE_UP, self.gate_up), (down, H, I, 0, self.down)):
            size = kmr.kmr_packed_size(N, K)
            out = torch.empty((E, size), dtype=torch.uint8, device="cuda")
            for e in range(E):
                q = r.integers(0, 16, (N, K), dtype=np.uint8)
                if flags == kmr.KMR_PACK_GATE_UP:
                    q[:, eights] = 8
                s, z = (torch.from_numpy(np.ascontiguousarray(v[e], np.float32)).bfloat16() for v in (ss, zz))
                keep.append(moe.dense(q, s.float().numpy(), z.float().numpy()))
                kmr.kmr_pack_int4(torch.from_numpy(q).cuda(), s.cuda(), z.cuda(), N, K, 128, flags, out[e], size, True, torch.cuda.current_stream())
            packed.append(out)
        self.dev = kmr.Moe(*packed, E, H, I, 128, torch.cuda.current_stream())


def even(r, E, N, K):
    return r.uniform(0.002, 0.02, (E, N, K // 128)), r.standard_normal((E, N, K // 128)) * 0.005


def uneven_layer(torch, r, E, H, I, how, F):
    """Rows of unequal size.  "down": one row of down F times the others; "same": one row of gate, the same of up and one of down; "apart":
    gate's and up's are different rows; "lognormal": every row has a size of its own."""
    gs, gz = even(r, E, 2 * I, H)
    ds, dz = even(r, E, H, I)
    gf, df = np.ones((E, 2 * I, 1)), np.ones((E, H, 1))
    for e in range(E):
        if how == "lognormal":
            gf[e, :, 0], df[e, :, 0] = np.exp(F * r.standard_normal(2 * I)), np.exp(F * r.standard_normal(H))
        else:
            i = r.integers(0, I)
            if how != "down":
                gf[e, i] = gf[e, I + (i if how == "same" else (i + 5) % I)] = F
            df[e, r.integers(0, H)] = F
    return Layer(torch, r, H, I, (gs * gf, gz * gf), (ds * df, dz * df)), df[:, :, 0]


def run(torch, layer, x, ids, w, dtype):
    T, k = ids.shape
    n = kmr.kmr_moe_experts_workspace_size(layer.dev, dtype, T, k)
    ws = torch.full(((n + 3) // 4,), float("nan"), device="cuda")
    y = torch.full(x.shape, float("nan"), device="cuda", dtype=x.dtype)
    kmr.kmr_moe_experts(layer.dev, x, dtype, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), T, k, y, kmr.KMR_EPI_NONE, ws, n,
                        torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    return y.double().cpu().numpy()


def places(r, T, E, k):
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    return ids, r.uniform(0.2, 1.0, (T, k)).astype(np.float32)


def worst(got, want):
    return max(rel_l2(g, v) for g, v in zip(got, want))


def condition(layer, x, ids, w, want, size):
    """By how much an error of the gates and ups, each relative to the size |row * x| of its own terms, counts in each result: where one
    activation makes up a result, the cancellation in that activation's own sums does."""
    out = np.zeros(len(x))
    I = layer.shape[2]
    for t in range(len(x)):
        for e, wt in zip(ids[t], w[t]):
            gu, terms = layer.gate_up[e] @ x[t], np.sqrt(layer.gate_up[e] ** 2 @ x[t] ** 2)
            with np.errstate(over="ignore"):
                g, u, sig = gu[:I], gu[I:], 1 / (1 + np.exp(-gu[:I]))
            slope = sig * (1 + g * (1 - sig))
            sens = (slope * u * terms[:I]) ** 2 + (sig * g * terms[I:]) ** 2
            out[t] += wt ** 2 * (((layer.down[e] / size[:, None]) ** 2) @ sens).sum()
    return np.sqrt(out) / np.linalg.norm(want / size, axis=1)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("E,H,I,T,k", [(4, 2048, 768, 4, 2), (4, 2048, 768, 17, 3), (3, 4096, 2048, 33, 1), (4, 1024, 384, 300, 2),
                                       (8, 256, 384, 4096, 2)])
@pytest.mark.parametrize("how,F", [("same", 1), ("down", 32), ("down", 1024), ("same", 8), ("same", 32), ("apart", 32), ("same", 256),
                                   ("apart", 256), ("lognormal", 1.0)])
def test_rows_of_unequal_size(torch, E, H, I, T, k, how, F, dtype):
    """Large rows of an expert cost the other rows nothing.  (Columns are compared at the size of their largest row: of a result that one
    column makes up, that column's own cancellation would be all that counts.)"""
    r = np.random.default_rng(E * H + I + T)
    layer, df = uneven_layer(torch, r, E, H, I, how, F)
    x, xv = rounded(torch, r.standard_normal((T, H)), dtype)
    ids, w = places(r, T, E, k)
    got = run(torch, layer, x, ids, w, dtype)
    some = np.unique(np.r_[0:min(T, 24), r.integers(0, T, 40)])
    want = moe.experts(xv[some], ids[some], w[some], layer.gate_up, layer.down)
    size = df.max(0)
    # (rows of any size: columns of less weight than their largest row's average no roundings)
    tol = TOL[dtype] if how != "lognormal" or dtype == kmr.KMR_F32 else 2.0 ** -8 + 2.0 ** -10
    tol = tol + 2e-6 * np.maximum(0, condition(layer, xv[some], ids[some], w[some], want, size) - 1)
    for scale, columns in ((size, size > 0), (np.ones(H), size <= 1.0)):
        for t in range(len(some)):
            assert rel_l2((got[some[t]] / scale)[columns], (want[t] / scale)[columns]) <= tol[t]


@pytest.mark.parametrize("E,H,I,T,k", SHAPES)
def test_single_precision_in_every_shape(torch, E, H, I, T, k):
    r = np.random.default_rng(E + H + I + T)
    layer = Layer(torch, r, H, I, even(r, E, 2 * I, H), even(r, E, H, I))
    x, xv = rounded(torch, r.standard_normal((T, H)) * np.exp(r.standard_normal((T, 1))), kmr.KMR_F32)
    ids, w = (np.concatenate(v, 1) for v in zip(*[places(r, T, E, min(k - i, E)) for i in range(0, k, E)]))
    some = np.unique(r.integers(0, T, 48))
    want = moe.experts(xv[some], ids[some], w[some], layer.gate_up, layer.down)
    assert worst(run(torch, layer, x, np.ascontiguousarray(ids), np.ascontiguousarray(w), kmr.KMR_F32)[some], want) <= TOL[kmr.KMR_F32]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("x_size,w_size", [(1e-8, 2.0 ** 8), (1e-12, 2.0 ** 16), (1e6, 2.0 ** -12), (1e10, 2.0 ** -24), (3e-4, 2.0 ** -4), (1.0, 1.0)])
def test_inputs_and_weights_far_from_one(torch, T, x_size, w_size, dtype):
    """Sizes whose results are ordinary numbers of single precision keep all their bits."""
    r = np.random.default_rng(17)
    E, H, I, k = 4, 512, 384, 2
    gs, gz = even(r, E, 2 * I, H)
    ds, dz = even(r, E, H, I)
    layer = Layer(torch, r, H, I, (gs * w_size, gz * w_size), (ds * w_size, dz * w_size))
    x, xv = rounded(torch, r.standard_normal((T, H)) * x_size, dtype)
    ids, w = places(r, T, E, k)
    want = moe.experts(xv, ids, w, layer.gate_up, layer.down)
    assert 1e-30 < np.abs(want).max(1).min() and np.abs(want).max() < 1e30
    assert worst(run(torch, layer, x, ids, w, dtype), want) <= TOL[dtype]


@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("dtype,F", [(kmr.KMR_F32, 2.0 ** 10), (kmr.KMR_F32, 2.0 ** 14), (kmr.KMR_BF16, 2.0 ** 14), (kmr.KMR_BF16, 2.0 ** 26)])
def test_inputs_of_unequal_size(torch, T, dtype, F):
    """One input of every 128 some F times the others', of weights that are zero: the others keep their bits (they go down
    to 2^-3 of each other, and 1/F of that of the largest)."""
    r = np.random.default_rng(37)
    E, H, I, k = 4, 512, 384, 2
    (gs, gz), (ds, dz) = even(r, E, 2 * I, H), even(r, E, H, I)
    big = np.arange(5, H, 128)
    layer = Layer(torch, r, H, I, (gs, gz * 0), (ds, dz), big)
    a = r.uniform(0.25, 2.0, (T, H)) * r.choice([-1.0, 1.0], (T, H))
    a[:, big] *= F
    x, xv = rounded(torch, a, dtype)
    ids, w = places(r, T, E, k)
    want = moe.experts(xv, ids, w, layer.gate_up, layer.down)
    assert worst(run(torch, layer, x, ids, w, dtype), want) <= TOL[dtype]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("gate", [-12.0, -30.0, -60.0])
def test_gates_that_are_nearly_shut(torch, T, gate, dtype):
    """Activations many orders below their gates and ups keep their bits: silu(g) = g exp(g) for these, so an error of the gate
    counts |g| times its share."""
    r = np.random.default_rng(23)
    E, H, I, k = 4, 512, 384, 2
    gs, gz = even(r, E, 2 * I, H)
    gs[:, :I] *= 0.05
    gz[:, :I] = gate / H * (1 + 0.1 * r.standard_normal((E, I, 1)))
    ds, dz = even(r, E, H, I)
    layer = Layer(torch, r, H, I, (gs, gz), (ds, dz))
    x, xv = rounded(torch, r.uniform(0.5, 1.5, (T, H)), dtype)
    ids, w = places(r, T, E, k)
    want = moe.experts(xv, ids, w, layer.gate_up, layer.down)
    assert np.abs(want).max(1).min() > 1e-36
    assert worst(run(torch, layer, x, ids, w, dtype), want) <= TOL[dtype] + 2e-6 * 1.5 * abs(gate)


@pytest.mark.parametrize("T", [3, 70])
def test_scales_that_differ_within_a_row(torch, T):
    """Groups of a row whose scales lie up to 2^14 apart.  Of many tokens a weight is held to half of 2^-24 and its offset to as much, against a largest
    weight of 2^-8 or more: 2^-16 of the row's largest weight, which one of its G groups has at the least."""
    r = np.random.default_rng(29)
    E, H, I, k = 4, 512, 512, 2
    spread = lambda s: (s[0] * 2.0 ** -r.integers(0, 15, s[0].shape), s[1] * 0)  # noqa: E731
    layer = Layer(torch, r, H, I, spread(even(r, E, 2 * I, H)), spread(even(r, E, H, I)))
    x, xv = rounded(torch, r.standard_normal((T, H)), kmr.KMR_F32)
    ids, w = places(r, T, E, k)
    want = moe.experts(xv, ids, w, layer.gate_up, layer.down)
    tol = TOL[kmr.KMR_F32] if T == 3 else 3 * 2.0 ** -16 * (H / 128) ** 0.5
    assert worst(run(torch, layer, x, ids, w, kmr.KMR_F32), want) <= tol


# The adapters' fp32 sums.  v: runs of 32 inputs, in which the small terms come first and cost nothing, then 2 steps of the tensor cores that
# cut off some 2^-25 of the run's sum each; the runs of the warps and CTAs are added in fp32 (four additions of half a 2^-24 at the
# most, at random: 4e-8 rms).  The second product: the small terms first again, then rank / 16 steps of 2^-25.  The result's
# own rounding: 2^-25 rms.
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("T", [5, 700])
def test_adapters_to_the_last_bits(torch, T, rank):
    r = np.random.default_rng(rank + T)
    K, N, L = 256, 512, 3
    a = torch.from_numpy((r.standard_normal((L, rank, K)) * K ** -0.5).astype(np.float32)).bfloat16().cuda()
    b = torch.from_numpy((r.standard_normal((L, N, rank)) * 0.3).astype(np.float32)).bfloat16().cuda()
    x, xv = rounded(torch, r.standard_normal((T, K)), kmr.KMR_F32)
    ids = np.repeat(r.integers(0, L, T), 40)[:T].astype(np.int32)
    y = torch.full((T, N), float("nan"), device="cuda")
    kmr.kmr_lora_apply(kmr.Lora(a, b), x, None, y, kmr.KMR_F32, torch.from_numpy(ids).cuda(), T, K, N, torch.cuda.current_stream())
    assert kmr.kmr_last_device_error() == 0
    want = moe.adapters(xv, np.zeros((T, N)), ids, a.float().cpu().numpy(), b.float().cpu().numpy(), np.full(L, rank), np.ones(L))
    err = rel_l2(y.double().cpu().numpy(), want)
    assert err <= 2 * 2.0 ** -25 + 4e-8 + rank / 16 * 2.0 ** -25 + 2.0 ** -25


def test_weights_prepared_on_another_stream(torch):
    """The factors' memory belongs to the stream that fills them: work still queued on the current stream, on memory freed there, does not
    reach them."""
    r = np.random.default_rng(41)
    E, H, I, T = 2, 256, 256, 20
    layer = Layer(torch, r, H, I, even(r, E, 2 * I, H), even(r, E, H, I))
    x, xv = rounded(torch, r.standard_normal((T, H)), kmr.KMR_F32)
    ids, w = places(r, T, E, 1)
    want = moe.experts(xv, ids, w, layer.gate_up, layer.down)
    gate_up, down, factors = layer.dev.tensors
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        freed = [torch.empty(factors.numel(), dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda._sleep(20_000_000)                        # some 10 ms
        for f in freed:
            f.fill_(255)                                     # NaN
        del freed, f
        layer.dev = kmr.Moe(gate_up, down, E, H, I, 128, stream)
        torch.cuda.synchronize()
        assert worst(run(torch, layer, x, ids, w, kmr.KMR_F32), want) <= TOL[kmr.KMR_F32]
