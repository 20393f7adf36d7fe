"""Refusals of the router, the experts and the adapters: every check below runs on the host before any CUDA call."""
import ctypes
import os

import pytest

import int4_weight_only_group_gb300 as kmr

P = 16            # a pointer that no call gets to use


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kmr.library_path()):
        from int4_weight_only_group_gb300.build import build
        build()
    return kmr.lib()


ARGS = {
    "kmr_moe_route": dict(logits=P, dtype=0, T=4, E=16, k=4, renorm=1, ids=P, weights=P),
    "kmr_moe_experts": dict(moe=None, x=P, dtype=0, ids=P, weights=P, T=4, k=2, y=P, epi=0, ws=P, n=1 << 40),
    "kmr_lora_apply": dict(lora=None, x=P, base=P, y=P, dtype=0, ids=P, T=4, ldx=64, ldy=32),
}
MOE = dict(gate_up=P, down=P, experts=8, hidden=256, intermediate=128, group=128, factors=P)
LORA = dict(a=P, b=P, ranks=None, scales=None, adapters=3, inputs=64, outputs=32, max_rank=16)


def call(L, name, given=None, **kw):
    """One call with good arguments but for those given (and those of the weights)."""
    assert set(kw) <= set(ARGS[name]), kw
    args = {**ARGS[name], **kw}
    keep = None
    if name == "kmr_moe_experts" and given is not False:
        keep = kmr.MoeStruct(**{**MOE, **(given or {})})
        args["moe"] = ctypes.addressof(keep)
    if name == "kmr_lora_apply" and given is not False:
        keep = kmr.LoraStruct(**{**LORA, **(given or {})})
        args["lora"] = ctypes.addressof(keep)
    return getattr(L, name)(*args.values(), None)


@pytest.mark.parametrize("name,kw,code", [
    ("kmr_moe_route", dict(logits=None), -1), ("kmr_moe_route", dict(ids=None), -1), ("kmr_moe_route", dict(weights=None), -1),
    ("kmr_moe_route", dict(dtype=2), -1), ("kmr_moe_route", dict(logits=18), -1), ("kmr_moe_route", dict(ids=18), -1),
    ("kmr_moe_route", dict(logits=17, dtype=1), -1), ("kmr_moe_route", dict(T=0), -9), ("kmr_moe_route", dict(T=(1 << 20) + 1), -9),
    ("kmr_moe_route", dict(E=0), -2), ("kmr_moe_route", dict(E=1025), -2), ("kmr_moe_route", dict(k=0), -2),
    ("kmr_moe_route", dict(k=33, E=64), -2), ("kmr_moe_route", dict(k=5, E=4), -2),
    ("kmr_moe_experts", dict(x=None), -1), ("kmr_moe_experts", dict(ids=None), -1), ("kmr_moe_experts", dict(weights=None), -1),
    ("kmr_moe_experts", dict(y=None), -1), ("kmr_moe_experts", dict(ws=None), -1), ("kmr_moe_experts", dict(x=8), -1),
    ("kmr_moe_experts", dict(y=24), -1), ("kmr_moe_experts", dict(ws=8), -1), ("kmr_moe_experts", dict(ids=2), -1),
    ("kmr_moe_experts", dict(weights=6), -1), ("kmr_moe_experts", dict(dtype=-1), -1), ("kmr_moe_experts", dict(epi=2), -1),
    ("kmr_moe_experts", dict(T=0), -9), ("kmr_moe_experts", dict(T=(1 << 20) + 1), -9), ("kmr_moe_experts", dict(k=0), -2),
    ("kmr_moe_experts", dict(k=33), -2), ("kmr_moe_experts", dict(n=15), -8),
    ("kmr_lora_apply", dict(x=None), -1), ("kmr_lora_apply", dict(y=None), -1), ("kmr_lora_apply", dict(ids=None), -1),
    ("kmr_lora_apply", dict(x=8), -1), ("kmr_lora_apply", dict(base=8), -1), ("kmr_lora_apply", dict(y=4), -1),
    ("kmr_lora_apply", dict(ids=2), -1), ("kmr_lora_apply", dict(dtype=3), -1), ("kmr_lora_apply", dict(T=0), -9),
    ("kmr_lora_apply", dict(T=(1 << 20) + 1), -9), ("kmr_lora_apply", dict(ldx=56), -2), ("kmr_lora_apply", dict(ldx=68), -2),
    ("kmr_lora_apply", dict(ldy=24), -2), ("kmr_lora_apply", dict(ldy=36), -2),
])
def test_bad_arguments(L, name, kw, code):
    assert call(L, name, **kw) == code


@pytest.mark.parametrize("name,kw,code", [
    ("kmr_moe_experts", False, -1), ("kmr_moe_experts", dict(gate_up=None), -1), ("kmr_moe_experts", dict(down=None), -1),
    ("kmr_moe_experts", dict(gate_up=24), -1), ("kmr_moe_experts", dict(experts=0), -2), ("kmr_moe_experts", dict(experts=1025), -2),
    ("kmr_moe_experts", dict(hidden=192), -2), ("kmr_moe_experts", dict(hidden=8320), -2), ("kmr_moe_experts", dict(hidden=0), -2),
    ("kmr_moe_experts", dict(intermediate=64), -2), ("kmr_moe_experts", dict(intermediate=8320), -2),
    ("kmr_moe_experts", dict(group=64), -2), ("kmr_moe_experts", dict(factors=None), -1), ("kmr_moe_experts", dict(factors=8), -1),
    ("kmr_lora_apply", False, -1), ("kmr_lora_apply", dict(a=None), -1), ("kmr_lora_apply", dict(b=None), -1),
    ("kmr_lora_apply", dict(a=8), -1), ("kmr_lora_apply", dict(b=8), -1), ("kmr_lora_apply", dict(ranks=2), -1),
    ("kmr_lora_apply", dict(scales=2), -1), ("kmr_lora_apply", dict(adapters=0), -2), ("kmr_lora_apply", dict(inputs=40), -2),
    ("kmr_lora_apply", dict(inputs=0), -2), ("kmr_lora_apply", dict(outputs=24), -2), ("kmr_lora_apply", dict(outputs=0), -2),
    ("kmr_lora_apply", dict(max_rank=12), -2), ("kmr_lora_apply", dict(max_rank=0), -2), ("kmr_lora_apply", dict(max_rank=136), -2),
])
def test_bad_weights(L, name, kw, code):
    assert call(L, name, kw) == code


def test_prepare_and_factors(L):
    assert L.kmr_moe_prepare(None, None) == -1
    for kw, code in ((dict(gate_up=None), -1), (dict(factors=None), -1), (dict(hidden=100), -2), (dict(group=32), -2)):
        m = kmr.MoeStruct(**{**MOE, **kw})
        assert L.kmr_moe_prepare(ctypes.addressof(m), None) == code
    F = L.kmr_moe_factors_size
    assert F(3, 256, 128) == 3 * (2 * 128 + 256 + 3) * 4
    assert F(0, 256, 128) == F(1025, 256, 128) == F(3, 200, 128) == F(3, 256, 8320) == 0


def test_workspace_size(L):
    W = L.kmr_moe_experts_workspace_size
    m = kmr.MoeStruct(**MOE)
    a = ctypes.addressof(m)
    assert W(a, 0, 1, 2) > 0 and W(a, 1, 4096, 8) >= W(a, 1, 1, 8) > 0
    assert W(None, 0, 1, 2) == W(a, 2, 1, 2) == W(a, 0, 0, 2) == W(a, 0, 1, 33) == 0
    assert W(ctypes.addressof(kmr.MoeStruct(**{**MOE, "hidden": 200})), 0, 1, 2) == 0


@pytest.mark.parametrize("E,H,I", [(1, 128, 8192), (1, 8192, 128), (64, 2048, 768), (8, 4096, 4096)])
def test_workspace_for_more_tokens_does_for_fewer(L, E, H, I):
    m = kmr.MoeStruct(**{**MOE, "experts": E, "hidden": H, "intermediate": I})
    for dtype in (kmr.KMR_F32, kmr.KMR_BF16):
        for k in (1, 2, 8, 32):
            sizes = [L.kmr_moe_experts_workspace_size(ctypes.addressof(m), dtype, T, k) for T in (*range(1, 80), 1000, 1024, 1025, 40000, 1 << 20)]
            assert sizes[0] > 0 and sizes == sorted(sizes)


def test_binding_checks_the_weights(L):
    torch = pytest.importorskip("torch")
    gu, dn = kmr.kmr_packed_size(256, 256), kmr.kmr_packed_size(256, 128)
    good = torch.zeros((3, gu), dtype=torch.uint8), torch.zeros((3, dn), dtype=torch.uint8)
    for a, b, args in ((good[0], good[1], (4, 256, 128)), (good[0], good[1], (3, 256, 64)), (good[0], good[0], (3, 256, 128)),
                       (good[0].view(torch.int16), good[1], (3, 256, 128)), (good[0].t(), good[1], (3, 256, 128))):
        with pytest.raises(ValueError):
            kmr.Moe(a, b, *args)
    a, b = torch.zeros((2, 16, 64), dtype=torch.bfloat16), torch.zeros((2, 32, 16), dtype=torch.bfloat16)
    lora = kmr.Lora(a, b, None, torch.ones(2))
    assert (lora.adapters, lora.inputs, lora.outputs, lora.max_rank) == (2, 64, 32, 16)
    for bad in ((a, b[:1], None, None), (a, b[:, :, :8], None, None), (a, b, torch.zeros(3, dtype=torch.int32), None),
                (a, b, None, torch.ones(1)), (a.float(), b, None, None), (a, b, torch.zeros(2), None), (a.transpose(0, 1), b, None, None)):
        with pytest.raises(ValueError):
            kmr.Lora(*bad)


def test_binding_checks_the_types(L):
    """A tensor of another type, with gaps or of other strides is refused by name."""
    torch = pytest.importorskip("torch")
    f, h, i = torch.zeros(64), torch.zeros(64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.int32)
    lora = kmr.Lora(torch.zeros((2, 16, 64), dtype=torch.bfloat16), torch.zeros((2, 32, 16), dtype=torch.bfloat16))
    for args, name in (((h, 0, 1, 8, 2, 1, i, f), "logits"), ((f, 1, 1, 8, 2, 1, i, f), "logits"), ((f, 0, 1, 8, 2, 1, i.long(), f), "ids"),
                       ((f, 0, 1, 8, 2, 1, i, h), "weights"), ((f[::2], 0, 1, 8, 2, 1, i, f), "logits")):
        with pytest.raises(ValueError, match=name):
            kmr.kmr_moe_route(*args)
    for args, name in (((h, 0, i, f, 1, 2, f), "x"), ((f, 0, f, f, 1, 2, f), "ids"), ((f, 0, i, i, 1, 2, f), "weights"), ((f, 0, i, f, 1, 2, h), "y")):
        with pytest.raises(ValueError, match=name + " is torch"):
            kmr.kmr_moe_experts(0, *args, 0, P, 0)
    x, y, wide = torch.zeros((4, 64)), torch.zeros((4, 32)), torch.zeros((4, 96))
    for args, name in (((x.bfloat16(), y, y, 0, i, 4, 64, 32), "x is"), ((x, y.double(), y, 0, i, 4, 64, 32), "base is"),
                       ((x, y, y, 0, i.long(), 4, 64, 32), "adapter_ids is"), ((x, y, wide[:, :32], 0, i, 4, 64, 32), "y has rows 96"),
                       ((x[:, ::2], y, y, 0, i, 4, 64, 32), "x has rows")):
        with pytest.raises(ValueError, match=name):
            kmr.kmr_lora_apply(lora, *args)
    with pytest.raises(kmr.KmrError) as e:                        # the right types go through to the library's checks
        kmr.kmr_lora_apply(lora, x, wide[:, :32], wide[:, 64:], 0, i, 0, 64, 96)
    assert e.value.code in (kmr.KMR_ERR_BATCH, kmr.KMR_ERR_INVALID_ARG)
