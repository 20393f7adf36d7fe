"""Products whose weights each token chooses: measured cases, their plain forms and their definition in 64 bits.

  route    a router's logits to each token's top-k experts and their weights
  experts  y[t] = sum_j weights[t, j] * down_e(silu(gate_e x[t]) * up_e x[t]), e = ids[t, j], over int4 group-wise
           experts (w = (q - 8) s + z, bf16 s and z per 128 inputs); an id of -1 is an unused place
  lora     y[t] = base[t] + scale_a * B_a (A_a x[t]) with the adapter a of the token's request, beside a shared
           projection's output; an adapter of -1 leaves base
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 128


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding sequence: latency
        {"name": "route, one token", "op": "route", "T": 1, "E": 128, "k": 8, "renorm": True, "bf16": False, "mask": False},
        # a batch of prompts; experts that are switched off, and padding whose mask leaves no expert
        {"name": "route, 4099 tokens of 60 experts", "op": "route", "T": 4099, "E": 60, "k": 4, "renorm": False, "bf16": True, "mask": True},
        # one decoding sequence through a 2048-wide layer of 128 small experts: latency
        {"name": "experts, one token", "op": "experts", "T": 1, "E": 128, "k": 8, "H": 2048, "I": 768, "bf16": False, "pad": 0},
        # the widest decode batch of the step
        {"name": "experts, 16 rows", "op": "experts", "T": 16, "E": 128, "k": 8, "H": 2048, "I": 768, "bf16": False, "pad": 0},
        # many decoding sequences padded to a captured batch, fewer and wider experts
        {"name": "experts, 61 rows of 80", "op": "experts", "T": 80, "E": 60, "k": 4, "H": 2048, "I": 1408, "bf16": True, "pad": 19},
        # a prompt in single precision
        {"name": "experts, prompt of 509", "op": "experts", "T": 509, "E": 128, "k": 8, "H": 2048, "I": 768, "bf16": False, "pad": 0},
        # a prompt through a few experts as wide as the dense layer
        {"name": "experts, 1024 tokens of 8 wide", "op": "experts", "T": 1024, "E": 8, "k": 2, "H": 2048, "I": 6144, "bf16": True, "pad": 0},
        # a chunk of prompts
        {"name": "experts, 4096 tokens", "op": "experts", "T": 4096, "E": 128, "k": 8, "H": 2048, "I": 768, "bf16": True, "pad": 0},
        # one decoding sequence with its adapter on the fused QKV projection
        {"name": "lora, one row", "op": "lora", "T": 1, "K": 2048, "N": 4096, "r": 16, "L": 8, "runs": 1, "bf16": False, "none": 0.0},
        # sixteen requests with their own adapters on the O projection, some with none
        {"name": "lora, 16 requests", "op": "lora", "T": 16, "K": 2048, "N": 2048, "r": 64, "L": 32, "runs": 16, "bf16": False, "none": 0.2},
        # prompts of nine requests in one chunk
        {"name": "lora, 9 prompts of 4077 rows", "op": "lora", "T": 4077, "K": 2048, "N": 4096, "r": 16, "L": 16, "runs": 9, "bf16": True, "none": 0.1},
        # a long chunk through the down projection's adapters, in single precision
        {"name": "lora, 8192 rows, down", "op": "lora", "T": 8192, "K": 6144, "N": 2048, "r": 32, "L": 4, "runs": 5, "bf16": False, "none": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "lora"])
    bf16 = rng.random() < 0.5
    if op == "route":
        E = _log(rng, 2, 512)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 10)), "renorm": rng.random() < 0.5,
                "bf16": bf16, "mask": rng.random() < 0.5}
    if op == "experts":
        E = rng.choice([1, 4, 8, 16, 60, 64, 128])
        H = 128 * rng.choice([2, 4, 8, 11, 16, 16, 20, 32])
        most = 600_000_000 // (E * 3 * H * 128)               # 600 million weights at the most
        I = 128 * _log(rng, 1, max(1, min(48, most)))
        k = rng.randint(1, min(E, 8))
        T = _log(rng, 1, max(1, min(4096, 300_000_000_000 // (6 * H * I * k))))
        return {"op": op, "T": T, "E": E, "k": k, "H": H, "I": I, "bf16": bf16, "pad": rng.choice([0, 0, rng.randint(0, T - 1)])}
    T = 1 if rng.random() < 0.2 else _log(rng, 2, 8192)
    K, N = 128 * _log(rng, 2, 48), 16 * _log(rng, 4, 400)
    runs = T if T <= 64 and rng.random() < 0.6 else _log(rng, 1, min(T, 32))
    return {"op": op, "T": T, "K": K, "N": N, "r": rng.choice([8, 16, 16, 32, 64, 128]), "L": _log(rng, 1, 64), "runs": runs,
            "bf16": bf16, "none": rng.choice([0.0, 0.0, 0.2])}


# ------------------------------------------------------------------ inputs
def _bf16(gen, shape, lo=None, hi=None, std=1.0):
    t = torch.rand(shape, generator=gen, device=DEV) * (hi - lo) + lo if lo is not None else torch.randn(shape, generator=gen, device=DEV) * std
    return t.bfloat16()


def _linear(gen, E, N, K):
    """E int4 matrices [N, K]: codes, scales and zeros."""
    q = torch.randint(0, 16, (E, N, K), generator=gen, device=DEV, dtype=torch.uint8)
    return q, _bf16(gen, (E, N, K // GROUP), 0.002, 0.02), _bf16(gen, (E, N, K // GROUP), std=0.005)


def _packed(lin, flags):
    import int4_weight_only_group_gb300 as kmr
    q, s, z = lin
    E, N, K = q.shape
    size = kmr.kmr_packed_size(N, K, GROUP)
    out = torch.empty((E, size), dtype=torch.uint8, device=DEV)
    for e in range(E):
        kmr.kmr_pack_int4(q[e], s[e], z[e], N, K, GROUP, flags, out[e], size, True, torch.cuda.current_stream())
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, T = case["op"], case["T"]
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    st = {"case": case}
    if op == "route":
        E, k = case["E"], case["k"]
        # some experts are liked by most tokens
        logits = 1.5 * torch.randn((T, E), generator=gen, device=DEV) + torch.randn(E, generator=gen, device=DEV)
        if case["mask"]:
            off = torch.rand(E, generator=gen, device=DEV) < 0.1
            logits[:, off] = -math.inf
            logits[torch.rand(T, generator=gen, device=DEV) < 0.05] = -math.inf
        st["logits"] = logits.to(dt)
        st["ids"] = torch.zeros((T, k), dtype=torch.int32, device=DEV)
        st["weights"] = torch.zeros((T, k), device=DEV)
    elif op == "experts":
        E, k, H, I = case["E"], case["k"], case["H"], case["I"]
        logits = 1.5 * torch.randn((T, E), generator=gen, device=DEV) + 0.7 * torch.randn(E, generator=gen, device=DEV)
        top = torch.topk(torch.softmax(logits, -1), k, dim=-1)
        there = torch.arange(T, device=DEV)[:, None] < T - case["pad"]
        st["ids"] = torch.where(there, top.indices, -1).to(torch.int32).contiguous()
        st["weights"] = torch.where(there, top.values / top.values.sum(-1, keepdim=True), 0.0).contiguous()
        st["x"] = torch.randn((T, H), generator=gen, device=DEV).to(dt)
        st["y"] = torch.zeros((T, H), dtype=dt, device=DEV)
        st["gate_up"], st["down"] = _linear(gen, E, 2 * I, H), _linear(gen, E, H, I)
        if own:
            import int4_weight_only_group_gb300 as kmr
            gate_up, down = _packed(st.pop("gate_up"), kmr.KMR_PACK_GATE_UP), _packed(st.pop("down"), 0)
            st["moe"] = kmr.Moe(gate_up, down, E, H, I, GROUP, torch.cuda.current_stream())
            st["dtype"] = kmr.KMR_BF16 if case["bf16"] else kmr.KMR_F32
            st["bytes"] = kmr.kmr_moe_experts_workspace_size(st["moe"], st["dtype"], T, k)
            st["ws"] = torch.empty(st["bytes"], dtype=torch.uint8, device=DEV)
    else:
        K, N, r, L, runs = case["K"], case["N"], case["r"], case["L"], case["runs"]
        st["a"], st["b"] = _bf16(gen, (L, r, K), std=K ** -0.5), _bf16(gen, (L, N, r), std=0.3)
        st["scales"] = torch.rand(L, generator=gen, device=DEV) * 2 + 0.25
        # each request: a run of rows with one adapter; lengths differ
        cut = torch.sort(torch.randperm(T - 1, generator=gen, device=DEV)[: runs - 1] + 1).values if runs > 1 else torch.empty(0, device=DEV)
        request = torch.searchsorted(cut.float(), torch.arange(T, device=DEV).float(), right=True)
        adapter = torch.randint(0, L, (runs,), generator=gen, device=DEV)
        adapter = torch.where(torch.rand(runs, generator=gen, device=DEV) < case["none"], -1, adapter)
        st["ids"] = adapter[request].to(torch.int32)
        st["x"] = torch.randn((T, K), generator=gen, device=DEV).to(dt)
        st["base"] = (2.0 * torch.randn((T, N), generator=gen, device=DEV)).to(dt)
        st["y"] = torch.zeros((T, N), dtype=dt, device=DEV)
        if own:
            import int4_weight_only_group_gb300 as kmr
            st["lora"] = kmr.Lora(st["a"], st["b"], None, st["scales"])
            st["dtype"] = kmr.KMR_BF16 if case["bf16"] else kmr.KMR_F32
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return {"route": _route, "experts": _experts, "lora": _lora}[st["case"]["op"]](st)


def _route(st):
    c = st["case"]
    if own:
        import int4_weight_only_group_gb300 as kmr
        kmr.kmr_moe_route(st["logits"], kmr.KMR_BF16 if c["bf16"] else kmr.KMR_F32, c["T"], c["E"], c["k"], c["renorm"], st["ids"],
                          st["weights"], torch.cuda.current_stream())
        return [st["ids"], st["weights"]]
    a = st["logits"].float()
    order = torch.argsort(a, dim=-1, descending=True, stable=True)[:, :c["k"]]
    top = a.gather(-1, order)
    real = top > -math.inf
    most = a.amax(-1, keepdim=True)
    most = torch.where(most > -math.inf, most, 0.0)
    e = torch.exp(top - most)
    total = e.sum(-1, keepdim=True) if c["renorm"] else torch.exp(a - most).sum(-1, keepdim=True)
    return [torch.where(real, order, -1).to(torch.int32), torch.where(real, e / total, 0.0)]


def _dense(lin, e):
    q, s, z = (t[e] for t in lin)
    w = (q.float().unflatten(-1, (-1, GROUP)) - 8.0) * s.float()[..., None] + z.float()[..., None]
    return w.flatten(-2)


def _experts(st):
    c = st["case"]
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
    if own:
        import int4_weight_only_group_gb300 as kmr
        kmr.kmr_moe_experts(st["moe"], st["x"], st["dtype"], st["ids"], st["weights"], T, k, st["y"], kmr.KMR_EPI_NONE, st["ws"],
                            st["bytes"], torch.cuda.current_stream())
        return [st["y"]]
    x = st["x"].float()
    place = torch.argsort(st["ids"].flatten(), stable=True)             # places in order of their expert
    count = torch.bincount(st["ids"].flatten() + 1, minlength=E + 1).tolist()
    out = torch.zeros((T * k, H), device=DEV)
    at = count[0]
    for e in range(E):
        if count[e + 1] == 0:
            continue
        mine = place[at:at + count[e + 1]]
        at += count[e + 1]
        h = torch.matmul(x[torch.div(mine, k, rounding_mode="floor")], _dense(st["gate_up"], e).T)
        h = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
        out[mine] = torch.matmul(h, _dense(st["down"], e).T)
    y = (out.view(T, k, H) * st["weights"][..., None]).sum(1)
    return [y.to(st["x"].dtype)]


def _lora(st):
    c = st["case"]
    T, K, N = c["T"], c["K"], c["N"]
    if own:
        import int4_weight_only_group_gb300 as kmr
        # fp32 rows are added to in place, as the plain form adds to them; bf16 ones go to rows of their own
        y = st["y"] if c["bf16"] else st["base"]
        kmr.kmr_lora_apply(st["lora"], st["x"], st["base"], y, st["dtype"], st["ids"], T, K, N, torch.cuda.current_stream())
        return [y]
    y = st["base"].float()
    x = st["x"].float()
    for a in torch.unique(st["ids"]).tolist():
        if a >= 0:
            rows = torch.nonzero(st["ids"] == a)[:, 0]
            v = torch.matmul(x[rows], st["a"][a].float().T)
            y[rows] += torch.matmul(v, st["b"][a].float().T) * st["scales"][a]
    return [y.to(st["x"].dtype)]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, T = case["op"], case["T"]
    size = 2 if case["bf16"] else 4
    if op == "route":
        return {"bytes": T * (case["E"] * size + 8 * case["k"]), "flops": T * case["E"] * 4}
    if op == "experts":
        E, k, H, I = case["E"], case["k"], case["H"], case["I"]
        rows = (T - case["pad"]) * k
        used = min(rows, E * (1.0 - (1.0 - k / E) ** (T - case["pad"])))   # experts that a token is sent to, if all are liked alike
        return {"bytes": used * 3 * H * I * (0.5 + 4 / GROUP) + T * (2 * H * size + 8 * k), "flops": 6 * rows * H * I}
    K, N, r = case["K"], case["N"], case["r"]
    used = min(case["L"] * (1.0 - (1.0 - 1.0 / case["L"]) ** case["runs"]), case["runs"]) * (1.0 - case["none"])
    return {"bytes": T * ((1.0 - case["none"]) * K + 2 * N) * size + 4 * T + used * r * (K + N) * 2,
            "flops": 2 * T * (1.0 - case["none"]) * r * (K + N)}


# ------------------------------------------------------------------ the definition in 64 bits
def _matrix64(lin, e):
    q, s, z = lin
    rep = lambda t: torch.repeat_interleave(t[e].double(), GROUP, dim=1)  # noqa: E731
    return (q[e].double() - 8) * rep(s) + rep(z)


def exact(case, seed):
    global own
    was, own = own, False                       # the unpacked weights
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, T = case["op"], case["T"]
    if op == "route":
        a = st["logits"].double().cpu()
        k = case["k"]
        p = torch.softmax(a, -1)
        w = torch.zeros((T, k), dtype=torch.float64)
        for t in range(T):
            row = a[t].tolist()
            top = [i for i in sorted(range(len(row)), key=lambda i: (-row[i], i))[:k] if row[i] > -math.inf]
            if top:
                v = p[t, top]
                w[t, :len(top)] = v / v.sum() if case["renorm"] else v
        return [None, w.to(DEV)]
    if op == "experts":
        k, I = case["k"], case["I"]
        x, y = st["x"].double(), torch.zeros(st["x"].shape, dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            share = torch.where(st["ids"] == e, st["weights"].double(), 0.0).sum(1)
            rows = torch.nonzero((st["ids"] == e).any(1)).flatten()
            if len(rows):
                gu = x[rows] @ _matrix64(st["gate_up"], e).mT
                act = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
                y[rows] += share[rows, None] * (act @ _matrix64(st["down"], e).mT)
        return [y]
    y = st["base"].double()
    for t0 in range(0, T, 1024):
        ids = st["ids"][t0:t0 + 1024]
        for a in sorted(set(ids.tolist()) - {-1}):
            delta = (st["x"][t0:t0 + 1024].double() @ st["a"][a].double().mT) @ st["b"][a].double().mT
            y[t0:t0 + 1024] += (ids == a)[:, None] * st["scales"][a].double() * delta
    return [y]
