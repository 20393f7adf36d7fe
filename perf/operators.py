"""The 4-bit KV cache's operators: measured cases, their plain forms and their definition in 64 bits.

  append    raw QKV rows of new tokens: per-head RMSNorm, 3-section M-RoPE, 4-bit K and V into the
            cache, rotated queries out
  convert   spans of a bf16 cache into the 4-bit cache, and back
  attn      decode attention of one token per row over the 4-bit cache, with or without adding every
            position's softmax weight to a running mass
  evict     the newest positions and the heaviest older ones of each row and head, compacted into
            another cache

Cache layout (head size d, nb = d / 32 blocks of 32 dims, group g): codes uint8 [slots][n_kv][max_len][d / 2],
low nibble first.  K row: [4][nb][8] nibbles, dim 32 b + 8 t + i at [t][b][i].  V row: [8][nb][4] nibbles, dim
32 b + 4 u + j at [u][b][j].  Scales int32 [slots][n_kv][max_len][d / g]: bf16 z in the low half, bf16 s in the
high half.  Value = code * s + z.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1e6
SECTIONS = {64: (8, 12, 12), 128: (16, 24, 24)}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one sequence through the 2B-shaped attention (16 query / 8 KV heads of 128): latency
        {"name": "append, one token", "op": "append", "B": 1, "T": 1, "nq": 16, "nkv": 8, "d": 128, "g": 32, "S": 1024, "ragged": False},
        # four prompts of different lengths, padded to the longest, appended to slots that hold a cached prefix
        {"name": "append, 4 ragged prompts", "op": "append", "B": 4, "T": 509, "nq": 16, "nkv": 8, "d": 128, "g": 64, "S": 1024, "ragged": True},
        # one long prompt into an empty slot
        {"name": "append, prompt of 8192", "op": "append", "B": 1, "T": 8192, "nq": 16, "nkv": 8, "d": 128, "g": 32, "S": 8192, "ragged": False},
        # a prefilled row of the tiny decoder (2 KV heads of 64) moved to 4 bits and read back
        {"name": "convert, 97 positions", "op": "convert", "B": 1, "T": 97, "nkv": 2, "d": 64, "g": 64, "S": 128, "ragged": False},
        # sixteen prefilled slots of up to 8192 positions
        {"name": "convert, 16 rows of 8192", "op": "convert", "B": 16, "T": 8192, "nkv": 8, "d": 128, "g": 32, "S": 8192, "ragged": True},
        # the 2B-shaped layer's decode at 600 cached positions
        {"name": "attn, 1 row of 601", "op": "attn", "B": 1, "L": 601, "nq": 16, "nkv": 8, "d": 128, "g": 32, "S": 1024, "mass": False, "ragged": False},
        # four continuous slots of different lengths, gathering the mass that eviction reads
        {"name": "attn, 4 slots, mass", "op": "attn", "B": 4, "L": 901, "nq": 16, "nkv": 8, "d": 128, "g": 32, "S": 1024, "mass": True, "ragged": True},
        # a wide batch of eight query heads per KV head, small heads
        {"name": "attn, 7 rows, 8 heads share", "op": "attn", "B": 7, "L": 4093, "nq": 32, "nkv": 4, "d": 64, "g": 64, "S": 4096, "mass": False, "ragged": True},
        # the sweep's largest point: 16 rows of 8192
        {"name": "attn, 16 rows of 8192", "op": "attn", "B": 16, "L": 8192, "nq": 16, "nkv": 8, "d": 128, "g": 32, "S": 8192, "mass": False, "ragged": False},
        # one very long context, with the mass
        {"name": "attn, 1 row of 131072, mass", "op": "attn", "B": 1, "L": 131072, "nq": 16, "nkv": 8, "d": 128, "g": 128, "S": 131072, "mass": True, "ragged": False},
        # one full slot cut to half
        {"name": "evict, 1024 to 512", "op": "evict", "B": 1, "n": 1024, "keep": 512, "recent": 64, "nkv": 8, "d": 128, "g": 32, "S": 1024, "ragged": False},
        # sixteen long slots of different lengths cut to 2048 positions
        {"name": "evict, 16 rows to 2048", "op": "evict", "B": 16, "n": 8192, "keep": 2048, "recent": 127, "nkv": 8, "d": 128, "g": 32, "S": 8192, "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "convert", "attn", "attn", "evict"])
    d = rng.choice([64, 128, 128])
    g = rng.choice([x for x in (32, 64, 128) if x <= d])
    nkv = rng.choice([1, 2, 4, 8, 8])
    rep = rng.choice([1, 2, 2, 3, 4, 6, 8])
    ragged = rng.random() < 0.6
    up = lambda v: (v + 15) // 16 * 16  # noqa: E731
    if op == "append":
        T = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        B = _log(rng, 1, max(1, min(64, 8192 // T)))
        rep = min(rep, 4)
        return {"op": op, "B": B, "T": T, "nq": nkv * rep, "nkv": nkv, "d": d, "g": g, "S": up(T + rng.randint(0, 1000)), "ragged": ragged}
    if op == "convert":
        T = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(16, 100000 // T)))
        return {"op": op, "B": B, "T": T, "nkv": nkv, "d": d, "g": g, "S": up(T + rng.randint(0, 300)), "ragged": ragged}
    if op == "attn":
        L = _log(rng, 1, 60000)
        B = _log(rng, 1, max(1, min(32, 100000 // L)))
        return {"op": op, "B": B, "L": L, "nq": nkv * rep, "nkv": nkv, "d": d, "g": g, "S": up(L + rng.randint(0, 300)), "mass": rng.random() < 0.5, "ragged": ragged}
    n = _log(rng, 16, 32768)
    B = _log(rng, 1, max(1, min(16, 100000 // n)))
    keep = rng.randint(1, n)
    return {"op": op, "B": B, "n": n, "keep": keep, "recent": rng.randint(0, keep), "nkv": nkv, "d": d, "g": g, "S": up(n + rng.randint(0, 300)), "ragged": ragged}


# ------------------------------------------------------------------ the 4-bit format, plain
def _quantize(x, g):
    """x fp32 [..., d] -> codes [..., d] and s, z [..., d / g] (fp32 values that bf16 holds)."""
    y = x.unflatten(-1, (-1, g))
    lo, hi = y.amin(-1), y.amax(-1)
    s = ((hi - lo) / torch.full_like(hi, 15.0)).bfloat16().float()
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    z = lo.bfloat16().float()
    c = torch.round((y - z[..., None]) / torch.where(s > 0, s, math.inf)[..., None]).clamp(0, 15)
    return c.flatten(-2), s, z


def _values(c, s, z, g):
    return (c.unflatten(-1, (-1, g)) * s[..., None] + z[..., None]).flatten(-2)


def _pack(c, key):
    """codes [..., d] -> the row's bytes [..., d / 2]."""
    d = c.shape[-1]
    c = c.to(torch.uint8)
    c = (c.unflatten(-1, (d // 32, 4, 8)) if key else c.unflatten(-1, (d // 32, 8, 4))).transpose(-3, -2).flatten(-3)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()


def _unpack(b, key):
    """the row's bytes [..., d / 2] -> codes fp32 [..., d]."""
    d = b.shape[-1] * 2
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    c = (c.unflatten(-1, (4, d // 32, 8)) if key else c.unflatten(-1, (8, d // 32, 4))).transpose(-3, -2).flatten(-3)
    return c.float()


def _bits(v):
    return v.bfloat16().view(torch.int16).to(torch.int32) & 0xFFFF


def _sz(s, z):
    return (_bits(z) | (_bits(s) << 16)).contiguous()


def _s_of(w):
    return (w & -65536).view(torch.float32)


def _z_of(w):
    return (w << 16).view(torch.float32)


# ------------------------------------------------------------------ inputs
def _lengths(case, gen, most):
    """One length per row: the longest row has `most`, the others anything from a third of it (ragged) or all of it."""
    B = case["B"]
    n = torch.full((B,), most, dtype=torch.int32, device=DEV)
    if case["ragged"] and B > 1:
        r = torch.rand(B, generator=gen, device=DEV)
        n = (most - (r * (most * 2 / 3))).int().clamp(min=1)
        n[-1] = most
    return n


def _cache(slots, nkv, S, d, g, gen, lengths, slot_ids):
    """A cache whose rows hold quantised N(0, 1) keys and values; positions past a row's length hold
    leftovers (random bytes, scales of NaN)."""
    out = {}
    n = torch.zeros(slots, dtype=torch.int32, device=DEV)
    n[slot_ids.long()] = lengths
    empty = torch.arange(S, device=DEV)[None, None, :, None] >= n[:, None, None, None]
    for name in ("k", "v"):
        codes = torch.empty((slots, nkv, S, d // 2), dtype=torch.uint8, device=DEV)
        sz = torch.empty((slots, nkv, S, d // g), dtype=torch.int32, device=DEV)
        for i in range(slots):
            c, s, z = _quantize(torch.randn((nkv, S, d), generator=gen, device=DEV), g)
            codes[i] = _pack(c, name == "k")
            sz[i] = torch.where(empty[i], torch.full_like(s, 0x7FC07FC0, dtype=torch.int32), _sz(s, z))
        out[name] = codes
        out[name + "_sz"] = sz
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, B, nkv, d, g, S = case["op"], case["B"], case["nkv"], case["d"], case["g"], case["S"]
    st = {"case": case}
    slots = B + 1
    st["slots"] = (torch.randperm(slots, generator=gen, device=DEV)[:B]).to(torch.int32)
    st["rows"] = torch.arange(B, dtype=torch.int32, device=DEV)
    st["zero"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if op == "append":
        T, nq = case["T"], case["nq"]
        st["n"] = _lengths(case, gen, T)
        st["cpos"] = (torch.rand(B, generator=gen, device=DEV) * (S - T + 1)).to(torch.int32).clamp(max=S - T)
        st["qkv"] = torch.randn((B, T, (nq + 2 * nkv) * d), generator=gen, device=DEV) * 2.0
        # image tokens: the height and width ids run apart from the time ids; far positions among them
        base = st["cpos"][:, None] + torch.arange(T, dtype=torch.int32, device=DEV)
        off = torch.randint(-40, 4000, (3, B, 1), generator=gen, device=DEV, dtype=torch.int32)
        st["pos"] = (base[None] + off).to(torch.int32).contiguous()
        st["wq"] = (1.0 + 0.1 * torch.randn(d, generator=gen, device=DEV)).bfloat16()
        st["wk"] = (1.0 + 0.1 * torch.randn(d, generator=gen, device=DEV)).bfloat16()
        st["q"] = torch.zeros((B, T, nq, d), device=DEV)
        st["kv"] = [torch.zeros((B, nkv, T, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        c = {}
        for name in ("k", "v"):
            c[name] = torch.zeros((slots, nkv, S, d // 2), dtype=torch.uint8, device=DEV)
            c[name + "_sz"] = torch.zeros((slots, nkv, S, d // g), dtype=torch.int32, device=DEV)
        st["cache"] = c
    elif op == "convert":
        T = case["T"]
        st["n"] = _lengths(case, gen, T)
        st["start"] = (torch.rand(B, generator=gen, device=DEV) * (S - T + 1)).to(torch.int32).clamp(max=S - T)
        st["src"] = [torch.randn((B, nkv, T, d), generator=gen, device=DEV).bfloat16() for _ in range(2)]
        st["kv"] = [torch.zeros((B, nkv, T, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        c = {}
        for name in ("k", "v"):
            c[name] = torch.zeros((slots, nkv, S, d // 2), dtype=torch.uint8, device=DEV)
            c[name + "_sz"] = torch.zeros((slots, nkv, S, d // g), dtype=torch.int32, device=DEV)
        st["cache"] = c
    elif op == "attn":
        nq = case["nq"]
        n = _lengths(case, gen, case["L"])
        st["cpos"] = n - 1
        st["cache"] = _cache(slots, nkv, S, d, g, gen, n, st["slots"])
        st["q"] = torch.randn((B, nq, d), generator=gen, device=DEV) * 1.5
        st["out"] = torch.zeros((B, nq, d), device=DEV)
        st["mass"] = torch.rand((slots, nkv, S), generator=gen, device=DEV) if case["mass"] else None
        if own:
            import int4_weight_only_group_gb300 as kmr
            h = _handle(st["cache"])
            st["ws_bytes"] = kmr.kmr_decode_attn_kv4_workspace_size(h, B, nq, case["mass"])
            st["ws"] = torch.empty(st["ws_bytes"], dtype=torch.uint8, device=DEV)
    else:
        n = _lengths(case, gen, case["n"])
        st["n"] = n
        st["cache"] = _cache(slots, nkv, S, d, g, gen, n, st["slots"])
        # heavy-tailed weights, and positions that were never attended
        m = torch.exp(2.0 * torch.randn((slots, nkv, S), generator=gen, device=DEV)) * 1e-2
        st["mass"] = torch.where(torch.rand((slots, nkv, S), generator=gen, device=DEV) < 0.2, torch.zeros_like(m), m)
        K = (case["keep"] + 15) // 16 * 16
        dst = {}
        for name in ("k", "v"):
            dst[name] = torch.zeros((B, nkv, K, d // 2), dtype=torch.uint8, device=DEV)
            dst[name + "_sz"] = torch.zeros((B, nkv, K, d // g), dtype=torch.int32, device=DEV)
        st["dst"] = dst
        st["dst_mass"] = torch.zeros((B, nkv, K), device=DEV)
        st["kept"] = torch.zeros((B, nkv, case["keep"]), dtype=torch.int32, device=DEV)
        st["new"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        st["kv"] = [torch.zeros((B, nkv, case["keep"], d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    if own:
        st["handle"] = _handle(st["cache"])
        if op == "evict":
            st["dst_handle"] = _handle(st["dst"])
    return st


def _handle(c):
    import int4_weight_only_group_gb300 as kmr
    return kmr.Kv4Cache(c["k"], c["v"], c["k_sz"], c["v_sz"])


# ------------------------------------------------------------------ one pass
def run(st):
    return {"append": _append, "convert": _convert, "attn": _attn, "evict": _evict}[st["case"]["op"]](st)


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, pos, d):
    """x fp32 [B, T, heads, d]; pos int32 [3, B, T]; the angles in 64 bits."""
    f = torch.arange(d // 2, device=x.device)
    a, b, _ = SECTIONS[d]
    axis = (f >= a).long() + (f >= a + b).long()
    ang = pos.double()[axis].permute(1, 2, 0) * torch.pow(torch.tensor(THETA, dtype=torch.float64, device=x.device), -2.0 * f.double() / d)
    cs, sn = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    lo, hi = x[..., : d // 2], x[..., d // 2:]
    return torch.cat((lo * cs - hi * sn, hi * cs + lo * sn), -1)


def _append(st):
    c = st["case"]
    B, T, nq, nkv, d, g = c["B"], c["T"], c["nq"], c["nkv"], c["d"], c["g"]
    if own:
        import int4_weight_only_group_gb300 as kmr
        stream = torch.cuda.current_stream()
        kmr.kmr_kv4_append(st["handle"], st["qkv"], st["pos"], st["slots"], st["cpos"], st["n"], B, T, nq, st["wq"], st["wk"],
                           EPS, THETA, SECTIONS[d], st["q"], None, stream)
        kmr.kmr_kv4_to_bf16(st["handle"], st["kv"][0], st["kv"][1], B, T, st["rows"], st["zero"], st["slots"], st["cpos"], st["n"], B, T, stream)
        return [st["q"], st["kv"][0], st["kv"][1]]
    x = st["qkv"].view(B, T, nq + 2 * nkv, d)
    there = (torch.arange(T, device=DEV)[None] < st["n"][:, None])[:, :, None, None]
    q = _rotate(_norm(x[:, :, :nq], st["wq"]), st["pos"], d)
    k = _rotate(_norm(x[:, :, nq:nq + nkv], st["wk"]), st["pos"], d)
    q = torch.where(there, q, st["q"])
    k = torch.where(there, _values(*_quantize(k, g), g), 0.0).transpose(1, 2).bfloat16()
    v = torch.where(there, _values(*_quantize(x[:, :, nq + nkv:], g), g), 0.0).transpose(1, 2).bfloat16()
    return [q, k, v]


def _convert(st):
    c = st["case"]
    B, T, g = c["B"], c["T"], c["g"]
    if own:
        import int4_weight_only_group_gb300 as kmr
        stream = torch.cuda.current_stream()
        kmr.kmr_kv4_from_bf16(st["handle"], st["src"][0], st["src"][1], B, T, st["rows"], st["zero"], st["slots"], st["start"], st["n"], B, T, stream)
        kmr.kmr_kv4_to_bf16(st["handle"], st["kv"][0], st["kv"][1], B, T, st["rows"], st["zero"], st["slots"], st["start"], st["n"], B, T, stream)
        return st["kv"]
    there = (torch.arange(T, device=DEV)[None] < st["n"][:, None])[:, None, :, None]
    k = torch.where(there, _values(*_quantize(st["src"][0].float(), g), g), 0.0).bfloat16()
    v = torch.where(there, _values(*_quantize(st["src"][1].float(), g), g), 0.0).bfloat16()
    return [k, v]


def _attn(st):
    c = st["case"]
    B, nq, nkv, d, g, L = c["B"], c["nq"], c["nkv"], c["d"], c["g"], c["L"]
    if own:
        import int4_weight_only_group_gb300 as kmr
        kmr.kmr_decode_attn_kv4(st["handle"], st["q"], st["slots"], st["cpos"], B, nq, 1.0 / math.sqrt(d), st["mass"], st["out"],
                                st["ws"], st["ws_bytes"], torch.cuda.current_stream())
        return [st["out"]] + ([st["mass"]] if c["mass"] else [])
    row = st["slots"].long()
    there = (torch.arange(L, device=DEV)[None] <= st["cpos"][:, None])[:, None, :]
    kw, vw = st["cache"]["k_sz"][row, :, :L], st["cache"]["v_sz"][row, :, :L]
    k = _values(_unpack(st["cache"]["k"][row, :, :L], True), _s_of(kw), _z_of(kw), g)
    k = torch.where(there[..., None], k, 0.0)
    a = torch.matmul(st["q"].view(B, nkv, nq // nkv, d), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    del k
    a = torch.where(there[:, :, None], a, -math.inf)
    p = torch.exp(a - a.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = _values(_unpack(st["cache"]["v"][row, :, :L], False), _s_of(vw), _z_of(vw), g)
    v = torch.where(there[..., None], v, 0.0)
    out = torch.matmul(p, v).view(B, nq, d)
    if not c["mass"]:
        return [out]
    st["mass"][:, :, :L].index_add_(0, row, p.sum(2))
    return [out, st["mass"]]


def _evict(st):
    c = st["case"]
    B, nkv, d, g, keep, recent, n = c["B"], c["nkv"], c["d"], c["g"], c["keep"], c["recent"], c["n"]
    if own:
        import int4_weight_only_group_gb300 as kmr
        stream = torch.cuda.current_stream()
        kmr.kmr_kv4_evict(st["handle"], st["dst_handle"], st["slots"], st["rows"], st["n"], B, keep, recent, st["mass"], st["dst_mass"],
                          st["kept"], st["new"], stream)
        kmr.kmr_kv4_to_bf16(st["dst_handle"], st["kv"][0], st["kv"][1], B, keep, st["rows"], st["zero"], st["rows"], st["zero"], st["new"], B, keep, stream)
        return [st["kept"], st["new"], st["dst_mass"], st["kv"][0], st["kv"][1]]
    row = st["slots"].long()
    at = torch.arange(n, device=DEV)[None, None]
    have = st["n"][:, None, None]
    mass = st["mass"][row, :, :n]
    rank = torch.where(at >= have, -math.inf, torch.where(at >= have - recent, math.inf, mass))
    kept = torch.argsort(rank, dim=-1, descending=True, stable=True)[..., :keep]
    kept = torch.where(kept < have, kept, n).sort(-1).values
    real = kept < n
    pick = torch.where(real, kept, 0)
    m = torch.zeros_like(st["dst_mass"])
    m[..., :keep] = torch.where(real, mass.gather(-1, pick), 0.0)
    out = []
    for name in ("k", "v"):
        w = st["cache"][name + "_sz"][row].gather(2, pick[..., None].expand(-1, -1, -1, d // g))
        b = st["cache"][name][row].gather(2, pick[..., None].expand(-1, -1, -1, d // 2))
        val = _values(_unpack(b, name == "k"), _s_of(w), _z_of(w), g)
        out.append(torch.where(real[..., None], val, 0.0).bfloat16())
    return [torch.where(real, kept, -1).to(torch.int32), st["n"].clamp(max=keep), m] + out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, B, nkv, d, g = case["op"], case["B"], case["nkv"], case["d"], case["g"]
    pos4 = nkv * 2 * (d // 2 + 4 * (d // g))       # a position of the 4-bit cache
    pos16 = nkv * 2 * 2 * d                        # the same position in bf16
    share = 2 / 3 if case["ragged"] and B > 1 else 1.0   # the mean length of ragged rows is about 2/3 of the longest
    if op == "append":
        tok, nq = B * case["T"] * share, case["nq"]
        # raw rows in, rotated queries and 4-bit K/V out; K/V read again and written as values
        return {"bytes": tok * (4 * (nq + 2 * nkv) * d + 4 * nq * d + 12 + 2 * pos4 + pos16), "flops": tok * (nq + 2 * nkv) * d * 12}
    if op == "convert":
        tok = B * case["T"] * share
        return {"bytes": tok * 2 * (pos4 + pos16), "flops": tok * nkv * d * 2 * 10}
    if op == "attn":
        tok, nq = B * case["L"] * share, case["nq"]
        return {"bytes": tok * (pos4 + (8 * nkv if case["mass"] else 0)) + B * nq * d * 8, "flops": tok * nq * d * 4}
    n, kept = B * case["n"] * share, B * min(case["keep"], case["n"] * share)
    return {"bytes": 4 * nkv * n + kept * (3 * pos4 + 8 * nkv + 4 * nkv + pos16), "flops": n * nkv * 4}


# ------------------------------------------------------------------ the definition in 64 bits
def _dims(row, key):
    """Codes of a cache row by dim, from the layout's byte and nibble addresses."""
    d = row.shape[-1] * 2
    nb = d // 32
    dim = torch.arange(d, device=row.device)
    b, r = dim // 32, dim % 32
    at = (r // 8) * nb * 8 + b * 8 + r % 8 if key else (r // 4) * nb * 4 + b * 4 + r % 4
    return (row[..., at // 2].long() >> (4 * (at % 2))) & 15


def _value64(row, word, key, g):
    d = row.shape[-1] * 2
    grp = torch.arange(d, device=row.device) // g
    as64 = lambda half: (half << 16).to(torch.int32).view(torch.float32).double()  # noqa: E731
    s, z = as64((word >> 16) & 0xFFFF), as64(word & 0xFFFF)
    return _dims(row, key).double() * s[..., grp] + z[..., grp]


def _quantized64(x, g):
    """The values that the 4-bit format holds for x (float64 [..., d])."""
    y = x.reshape(*x.shape[:-1], -1, g)
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    s = ((hi - lo) / 15).float().bfloat16().double()
    z = lo.float().bfloat16().double()
    c = torch.round((y - z) / s.clamp(min=2.0 ** -126)).clamp(0, 15)
    return (c * s + z).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op, B, nkv, d, g = case["op"], case["B"], case["nkv"], case["d"], case["g"]
    if op == "append":
        T, nq = case["T"], case["nq"]
        x = st["qkv"].double().reshape(B, T, -1, d)
        half = d // 2
        sec = torch.tensor(SECTIONS[d], device=DEV)
        axis = torch.repeat_interleave(torch.arange(3, device=DEV), sec)
        freq = torch.exp(torch.arange(half, device=DEV, dtype=torch.float64) * (-2.0 / d * math.log(THETA)))
        ang = torch.stack([st["pos"][int(axis[i])].double() * freq[i] for i in range(half)], -1)
        turn = torch.polar(torch.ones_like(ang), ang)[:, :, None]
        res = []
        for lo, hi, w in ((0, nq, st["wq"]), (nq, nq + nkv, st["wk"])):
            h = x[:, :, lo:hi]
            h = h / torch.sqrt((h * h).sum(-1, keepdim=True) / d + EPS) * w.double()
            zc = torch.complex(h[..., :half].contiguous(), h[..., half:].contiguous()) * turn
            res.append(torch.cat((zc.real, zc.imag), -1))
        gone = torch.arange(T, device=DEV)[None] >= st["n"][:, None]
        res[0][gone] = 0.0
        k, v = _quantized64(res[1], g), _quantized64(x[:, :, nq + nkv:], g)
        k[gone] = 0.0
        v[gone] = 0.0
        return [res[0], k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()]
    if op == "convert":
        out = []
        for src in st["src"]:
            val = _quantized64(src.double(), g)
            for b in range(B):
                val[b, :, int(st["n"][b]):] = 0.0
            out.append(val)
        return out
    if op == "attn":
        nq = case["nq"]
        out = torch.zeros((B, nq, d), dtype=torch.float64, device=DEV)
        mass = st["mass"].double() if case["mass"] else None
        for b in range(B):
            slot, n = int(st["slots"][b]), int(st["cpos"][b]) + 1
            for h in range(nkv):
                k = _value64(st["cache"]["k"][slot, h, :n], st["cache"]["k_sz"][slot, h, :n], True, g)
                v = _value64(st["cache"]["v"][slot, h, :n], st["cache"]["v_sz"][slot, h, :n], False, g)
                mine = slice(h * (nq // nkv), (h + 1) * (nq // nkv))
                p = torch.softmax(st["q"][b, mine].double() @ k.T / math.sqrt(d), -1)
                out[b, mine] = p @ v
                if mass is not None:
                    mass[slot, h, :n] += p.sum(0)
        return [out] + ([mass] if case["mass"] else [])
    keep, recent = case["keep"], case["recent"]
    kept = torch.full((B, nkv, keep), -1, dtype=torch.int64)
    mass = torch.zeros_like(st["dst_mass"], dtype=torch.float64)
    kv = [torch.zeros((B, nkv, keep, d), dtype=torch.float64, device=DEV) for _ in range(2)]
    for b in range(B):
        slot, n = int(st["slots"][b]), int(st["n"][b])
        for h in range(nkv):
            old = st["mass"][slot, h, :max(0, n - recent)].double().cpu().tolist()
            top = sorted(range(len(old)), key=lambda i: (-old[i], i))[:max(0, min(keep, n) - min(recent, n))]
            idx = torch.tensor(sorted(top) + list(range(max(0, n - recent), n)), dtype=torch.int64, device=DEV)
            kept[b, h, :len(idx)] = idx.cpu()
            mass[b, h, :len(idx)] = st["mass"][slot, h, idx].double()
            for o, name in ((0, "k"), (1, "v")):
                kv[o][b, h, :len(idx)] = _value64(st["cache"][name][slot, h, idx], st["cache"][name + "_sz"][slot, h, idx], name == "k", g)
    return [None, None, mass] + kv
