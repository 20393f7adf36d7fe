"""Refusals of the 4-bit cache's entry points: every check below runs on the host before any CUDA call."""
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


def cache(**kw):
    f = dict(k_codes=P, v_codes=P, k_sz=P, v_sz=P, slots=4, n_kv_heads=8, max_len=64, head_dim=128, group=32)
    f.update(kw)
    return kmr.Kv4CacheStruct(**f)


BAD_CACHES = [(dict(k_codes=None), kmr.KMR_ERR_INVALID_ARG), (dict(v_codes=None), kmr.KMR_ERR_INVALID_ARG),
              (dict(k_sz=None), kmr.KMR_ERR_INVALID_ARG), (dict(v_sz=None), kmr.KMR_ERR_INVALID_ARG),
              (dict(k_codes=24), kmr.KMR_ERR_INVALID_ARG), (dict(v_sz=4), kmr.KMR_ERR_INVALID_ARG),
              (dict(slots=0), kmr.KMR_ERR_SHAPE), (dict(n_kv_heads=0), kmr.KMR_ERR_SHAPE),
              (dict(n_kv_heads=1025), kmr.KMR_ERR_SHAPE), (dict(max_len=0), kmr.KMR_ERR_SHAPE),
              (dict(max_len=40), kmr.KMR_ERR_SHAPE), (dict(max_len=(1 << 28) + 16), kmr.KMR_ERR_SHAPE),
              (dict(head_dim=96), kmr.KMR_ERR_SHAPE), (dict(group=16), kmr.KMR_ERR_SHAPE),
              (dict(head_dim=64, group=128), kmr.KMR_ERR_SHAPE)]


def call(L, name, c, **kw):
    """One call with good arguments but for those given."""
    sec = (ctypes.c_int * 3)(*kw.pop("sections", (16, 24, 24)))
    base = {
        "kmr_kv4_append": dict(qkv=P, positions=P, slot_ids=P, cpos=P, n=None, B=2, T=1, nq=16, wq=P, wk=P, eps=1e-6,
                               theta=1e6, sec=sec, q=P, mass=None),
        "kmr_kv4_from_bf16": dict(k=P, v=P, slots16=2, len16=64, ids16=P, start16=P, ids=P, start=P, n=P, B=2, T=4),
        "kmr_kv4_to_bf16": dict(k=P, v=P, slots16=2, len16=64, ids16=P, start16=P, ids=P, start=P, n=P, B=2, T=4),
        "kmr_decode_attn_kv4": dict(q=P, ids=P, cpos=P, B=2, nq=16, scale=0.1, mass=None, out=P, ws=P, n=1 << 40),
        "kmr_kv4_evict": dict(dst=ctypes.addressof(c), ids=P, dids=P, n=P, B=2, keep=8, recent=2, mass=P, dmass=None,
                              kept=P, new=P),
    }[name]
    assert set(kw) <= set(base), kw
    base.update(kw)
    return getattr(L, name)(ctypes.addressof(c), *base.values(), None)


NAMES = ["kmr_kv4_append", "kmr_kv4_from_bf16", "kmr_kv4_to_bf16", "kmr_decode_attn_kv4", "kmr_kv4_evict"]


@pytest.mark.parametrize("name", NAMES)
def test_bad_caches(L, name):
    for kw, code in BAD_CACHES:
        assert call(L, name, cache(**kw)) == code, kw
    args = [0 if t in (ctypes.c_int, ctypes.c_float, ctypes.c_size_t) else None for t in getattr(L, name).argtypes]
    assert getattr(L, name)(*args) == kmr.KMR_ERR_INVALID_ARG


@pytest.mark.parametrize("name,kw,code", [
    ("kmr_kv4_append", dict(qkv=None), -1), ("kmr_kv4_append", dict(positions=None), -1),
    ("kmr_kv4_append", dict(slot_ids=None), -1), ("kmr_kv4_append", dict(cpos=None), -1),
    ("kmr_kv4_append", dict(sec=None), -1), ("kmr_kv4_append", dict(q=None), -1),
    ("kmr_kv4_append", dict(qkv=8), -1), ("kmr_kv4_append", dict(q=4), -1), ("kmr_kv4_append", dict(wq=2), -1),
    ("kmr_kv4_append", dict(eps=-1.0), -1), ("kmr_kv4_append", dict(eps=float("nan")), -1),
    ("kmr_kv4_append", dict(theta=0.0), -1), ("kmr_kv4_append", dict(theta=float("inf")), -1),
    ("kmr_kv4_append", dict(T=0), -1), ("kmr_kv4_append", dict(T=(1 << 28) + 1), -1), ("kmr_kv4_append", dict(B=0), -9), ("kmr_kv4_append", dict(B=1025), -9),
    ("kmr_kv4_append", dict(nq=12), -2), ("kmr_kv4_append", dict(nq=72), -2), ("kmr_kv4_append", dict(nq=0), -2),
    ("kmr_kv4_append", dict(sections=(16, 24, 23)), -2), ("kmr_kv4_append", dict(sections=(-16, 56, 24)), -2),
    ("kmr_kv4_from_bf16", dict(k=None), -1), ("kmr_kv4_from_bf16", dict(v=8), -1),
    ("kmr_kv4_from_bf16", dict(ids16=None), -1), ("kmr_kv4_from_bf16", dict(n=None), -1),
    ("kmr_kv4_from_bf16", dict(T=0), -1), ("kmr_kv4_from_bf16", dict(T=(1 << 31) - 1), -1), ("kmr_kv4_from_bf16", dict(B=0), -9),
    ("kmr_kv4_from_bf16", dict(slots16=0), -2), ("kmr_kv4_from_bf16", dict(len16=0), -2),
    ("kmr_kv4_to_bf16", dict(k=None), -1), ("kmr_kv4_to_bf16", dict(start=None), -1),
    ("kmr_kv4_to_bf16", dict(B=1025), -9), ("kmr_kv4_to_bf16", dict(T=-1), -1),
    ("kmr_decode_attn_kv4", dict(q=None), -1), ("kmr_decode_attn_kv4", dict(out=None), -1),
    ("kmr_decode_attn_kv4", dict(ws=None), -1), ("kmr_decode_attn_kv4", dict(q=8), -1), ("kmr_decode_attn_kv4", dict(mass=4), -1),
    ("kmr_decode_attn_kv4", dict(scale=float("nan")), -1), ("kmr_decode_attn_kv4", dict(scale=float("inf")), -1),
    ("kmr_decode_attn_kv4", dict(B=0), -9), ("kmr_decode_attn_kv4", dict(nq=20), -2),
    ("kmr_decode_attn_kv4", dict(nq=72), -2), ("kmr_decode_attn_kv4", dict(n=15), -8),
    ("kmr_kv4_evict", dict(dst=None), -1), ("kmr_kv4_evict", dict(ids=None), -1), ("kmr_kv4_evict", dict(dids=None), -1),
    ("kmr_kv4_evict", dict(n=None), -1), ("kmr_kv4_evict", dict(mass=None), -1), ("kmr_kv4_evict", dict(kept=None), -1),
    ("kmr_kv4_evict", dict(new=None), -1), ("kmr_kv4_evict", dict(keep=0), -1), ("kmr_kv4_evict", dict(recent=-1), -1),
    ("kmr_kv4_evict", dict(recent=9), -1), ("kmr_kv4_evict", dict(B=0), -9), ("kmr_kv4_evict", dict(keep=65), -4),
])
def test_bad_arguments(L, name, kw, code):
    assert call(L, name, cache(), **kw) == code


def test_evict_between_caches(L):
    for kw, code in ((dict(n_kv_heads=4), -2), (dict(head_dim=64), -2), (dict(group=64), -2), (dict(max_len=80), -2),
                     (dict(k_codes=32, group=64), -2)):
        other = cache(**kw)
        assert call(L, "kmr_kv4_evict", cache(), dst=ctypes.addressof(other)) == code, kw
    other = cache(k_codes=32, v_codes=32, k_sz=32, v_sz=32, max_len=16)
    assert call(L, "kmr_kv4_evict", cache(), dst=ctypes.addressof(other), keep=17) == kmr.KMR_ERR_CACHE_FULL
    assert call(L, "kmr_kv4_evict", cache(), dst=ctypes.addressof(other), dmass=P) == kmr.KMR_ERR_INVALID_ARG


def test_workspace_size(L):
    W = L.kmr_decode_attn_kv4_workspace_size
    c = cache(max_len=8192)
    a = ctypes.addressof(c)
    assert 0 < W(a, 1, 16, 0) < W(a, 4, 16, 0) and W(a, 1, 16, 1) == W(a, 1, 16, 0) + 16 * 8192 * 4
    assert W(a, 0, 16, 0) == W(a, 1, 12, 0) == W(a, 1025, 16, 0) == W(None, 1, 16, 0) == 0
    assert W(ctypes.addressof(cache(group=48)), 1, 16, 0) == 0
    assert W(ctypes.addressof(cache(max_len=2048)), 4, 16, 1) == 16           # short caches merge on chip


def test_binding_checks_the_cache_tensors(L):
    torch = pytest.importorskip("torch")
    c = kmr.Kv4Cache.zeros(2, 3, 32, 64, 32, device="cpu")
    assert (c.slots, c.n_kv_heads, c.max_len, c.head_dim, c.group) == (2, 3, 32, 64, 32)
    assert c.nbytes == 2 * 2 * 3 * 32 * (32 + 8)
    k, v, ks, vs = c.tensors
    for bad in ((k, v, ks[:, :, :16], vs), (k, v[:, :2], ks, vs), (k, v, ks.to(torch.int64), vs),
                (k.transpose(1, 2), v, ks, vs), (k, v, ks, vs.to(torch.int16))):
        with pytest.raises(ValueError):
            kmr.Kv4Cache(*bad)
    with pytest.raises(ValueError):
        kmr.kmr_kv4_append(c, 16, 16, 16, 16, None, 1, 1, 3, None, None, 1e-6, 1e6, (16, 16), 16)
    with pytest.raises(kmr.KmrError) as e:
        kmr.kmr_kv4_append(c, 16, 16, 16, 16, None, 1, 1, 3, None, None, 1e-6, 1e6, (16, 16, 1), 16)
    assert e.value.code == kmr.KMR_ERR_SHAPE


def test_evict_outputs_share_no_memory_with_what_is_read(L):
    """`lengths` cut in place, for instance: another head's CTAs would read the cut length.  4 rows, 8 heads, 8 kept."""
    at = dict(ids=0x1000, dids=0x2000, n=0x3000, kept=0x4000, new=0x5000, B=4)
    for kw in (dict(new=0x3000), dict(new=0x1000), dict(new=0x2000), dict(new=0x300C), dict(new=0x2FF4), dict(kept=0x3000),
               dict(kept=0x1004), dict(kept=0x2000), dict(kept=0x3000 - 4 * 8 * 8 * 4 + 4), dict(new=0x4000), dict(kept=0x500C),
               dict(new=0x4000 + 4 * 8 * 8 * 4 - 4)):
        assert call(L, "kmr_kv4_evict", cache(), **{**at, **kw}) == kmr.KMR_ERR_INVALID_ARG, kw


CALLS = {
    "kmr_kv4_append": ("qkv positions slot_ids cache_position n_tokens q_norm k_norm q_out mass",
                       lambda c, a: kmr.kmr_kv4_append(c, a["qkv"], a["positions"], a["slot_ids"], a["cache_position"], a["n_tokens"],
                                                       0, 3, 6, a["q_norm"], a["k_norm"], 1e-6, 1e6, (8, 12, 12), a["q_out"], a["mass"])),
    "kmr_kv4_from_bf16": ("k_bf16 v_bf16 bf16_slot_ids bf16_start slot_ids start lengths",
                          lambda c, a: kmr.kmr_kv4_from_bf16(c, a["k_bf16"], a["v_bf16"], 4, 20, a["bf16_slot_ids"], a["bf16_start"],
                                                             a["slot_ids"], a["start"], a["lengths"], 0, 5)),
    "kmr_kv4_to_bf16": ("k_bf16 v_bf16 bf16_slot_ids bf16_start slot_ids start lengths",
                        lambda c, a: kmr.kmr_kv4_to_bf16(c, a["k_bf16"], a["v_bf16"], 4, 20, a["bf16_slot_ids"], a["bf16_start"],
                                                         a["slot_ids"], a["start"], a["lengths"], 0, 5)),
    "kmr_decode_attn_kv4": ("q slot_ids cache_position mass out",
                            lambda c, a: kmr.kmr_decode_attn_kv4(c, a["q"], a["slot_ids"], a["cache_position"], 0, 6, 0.1, a["mass"],
                                                                 a["out"], 16, 16)),
    "kmr_kv4_evict": ("src_slot_ids dst_slot_ids lengths mass dst_mass kept new_lengths",
                      lambda c, a: kmr.kmr_kv4_evict(c, c, a["src_slot_ids"], a["dst_slot_ids"], a["lengths"], 0, 7, 2, a["mass"],
                                                     a["dst_mass"], a["kept"], a["new_lengths"])),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_binding_checks_the_types(L, name):
    """A tensor of another type (an int64 index, a bf16 query) or with gaps is refused by name; the right types go through
    to the library, which refuses the call for its batch of 0 before it looks at anything else."""
    torch = pytest.importorskip("torch")
    names, run = CALLS[name]
    cache_on = kmr.Kv4Cache.zeros(4, 3, 32, 64, 32, device="cpu")
    names = names.split()
    kinds = {k: torch.float32 if k in ("qkv", "q_out", "mass", "dst_mass", "q", "out") else
             torch.bfloat16 if k in ("q_norm", "k_norm", "k_bf16", "v_bf16") else torch.int32 for k in names}
    # (a tensor of its own for each: the library compares the addresses)
    good = {k: torch.zeros(64, dtype=kinds[k]) for k in names}
    others = {torch.float32: (torch.bfloat16, torch.float64, torch.int32), torch.int32: (torch.int64, torch.int16, torch.float32),
              torch.bfloat16: (torch.float16, torch.float32)}
    for key in names:
        for t in others[kinds[key]]:
            with pytest.raises(ValueError, match=key + " is torch"):
                run(cache_on, {**good, key: torch.zeros(64, dtype=t)})
        with pytest.raises(ValueError, match=key + " must be contiguous"):
            run(cache_on, {**good, key: torch.zeros(128, dtype=kinds[key])[::2]})
        with pytest.raises(TypeError, match=key):
            run(cache_on, {**good, key: "text"})
    for key in names:
        if kinds[key] == torch.bfloat16:                        # also as its bits
            good[key] = good[key].view(torch.int16)
    with pytest.raises(kmr.KmrError) as e:
        run(cache_on, good)
    assert e.value.code == kmr.KMR_ERR_BATCH
