"""The operators whose weights each row of a batch picks for itself, as work to be measured.

Three operators stand beside the packed linear in a serving stack:

  route    the router of a mixture of experts: scores, a bias for balance,
           groups, the best k experts a token and their weights
  experts  the gated linears of the experts a token picked, on packed int4
           weights (bf16 or int8 activations), summed with the router's weights
  lora     low-rank adapters of many requests at once, beside a shared
           projection: each token's adapter, added to the projection's output

`listed()` holds the cases, `draw(rng)` more of the same ranges, `prepare` makes
what a program has in hand, `run` is one pass. With `own` false a pass is the
operator's plain form in elementary torch operations in 32 bits; with `own` true
it is the call a user makes. `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

GROUP = 128      # weights of one row that share a scale and a zero point
DEV = "cuda"


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one token of a chat: a small softmax router, latency only
        dict(name="route-1", op="route", T=1, E=64, k=6, score="softmax", bias=False, groups=1,
             top_groups=1, top2=False, renorm=True, scale=1.0, dtype="bf16"),
        # a ragged prefill chunk, groups by their best expert, weights as they are
        dict(name="route-1037", op="route", T=1037, E=160, k=6, score="softmax", bias=False,
             groups=8, top_groups=3, top2=False, renorm=False, scale=16.0, dtype="bf16"),
        # the largest prefill batch: sigmoid scores, a balance bias, groups by
        # their two best experts, renormalised and scaled weights
        dict(name="route-16384", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, top2=True, renorm=True, scale=2.5, dtype="f32"),
        # one token through its experts: every weight byte is read once
        dict(name="experts-1", op="experts", variant="w4a16", T=1, E=64, k=8, H=3584, I=1280,
             dropped=0.0),
        # a decode batch of many requests: few tokens an expert
        dict(name="experts-33", op="experts", variant="w4a8", T=33, E=64, k=8, H=3584, I=1280,
             dropped=0.0),
        # a short prefill of a smaller layer; a quarter of the picks belong to
        # experts of another machine
        dict(name="experts-509", op="experts", variant="w4a16", T=509, E=32, k=4, H=2048, I=1024,
             dropped=0.25),
        # the largest prefill batch, int8 activations
        dict(name="experts-4096", op="experts", variant="w4a8", T=4096, E=64, k=8, H=3584, I=1280,
             dropped=0.0),
        # a ragged prefill batch, bf16 activations
        dict(name="experts-2977", op="experts", variant="w4a16", T=2977, E=64, k=6, H=2048, I=1408,
             dropped=0.0),
        # one token, one adapter of 32 (attention output projection)
        dict(name="lora-1", op="lora", fused=False, M=1, L=32, r=16, K=3584, N=3584, mixed=False),
        # a decode batch: many requests, adapters of several ranks, some without
        # one (gate / up projection)
        dict(name="lora-67", op="lora", fused=False, M=67, L=64, r=32, K=3584, N=18944, mixed=True),
        # a prefill batch of a few requests with adapters of a high rank
        dict(name="lora-4093", op="lora", fused=False, M=4093, L=8, r=64, K=3584, N=3584, mixed=True),
        # the whole W4A8 projection with its adapters in one call
        dict(name="lora-linear-256", op="lora", fused=True, M=256, L=16, r=16, K=3584, N=3584,
             mixed=True),
    ]


def draw(rng):
    """One more case of the ranges above (no name)."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["route", "experts", "lora"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, top_groups * (E // groups)))
        sig = rng.random() < 0.5
        return dict(op="route", T=log_int(1, 16384), E=E, k=k,
                    score="sigmoid" if sig else "softmax", bias=sig and rng.random() < 0.7,
                    groups=groups, top_groups=top_groups, top2=sig and groups > 1,
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                    dtype="f32" if sig and rng.random() < 0.5 else "bf16")
    if op == "experts":
        E = rng.choice([8, 16, 24, 32, 48, 64])
        return dict(op="experts", variant=rng.choice(["w4a16", "w4a8"]), T=log_int(1, 4096), E=E,
                    k=rng.randint(1, min(8, E)), H=128 * rng.randint(4, 28),
                    I=128 * rng.randint(2, 10), dropped=rng.choice([0.0, 0.0, 0.25]))
    fused = rng.random() < 0.3
    return dict(op="lora", fused=fused, M=log_int(1, 4096), L=rng.randint(1, 64),
                r=8 * rng.randint(1, 8), K=128 * rng.randint(4, 28),
                N=128 * rng.randint(4, 28 if fused else 148), mixed=rng.random() < 0.7)


# -------------------------------------------------------------------- work ---

def _touched(E, k, T):
    """Experts that T tokens of k picks each reach, on average."""
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    c = case
    if c["op"] == "route":
        nb = c["T"] * c["E"] * (2 if c["dtype"] == "bf16" else 4) + c["T"] * c["k"] * 8
        return {"bytes": nb + (4 * c["E"] if c["bias"] else 0), "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "experts":
        H, I, T = c["H"], c["I"], c["T"]
        rows = T * c["k"] * (1.0 - c["dropped"])
        weights = 3 * H * I * (0.5 + 2.5 / GROUP)
        touched = _touched(c["E"], c["k"] * (1.0 - c["dropped"]), T)
        return {"bytes": touched * weights + T * H * 4 + T * c["k"] * 8,
                "flops": 2.0 * rows * 3 * H * I}
    M, K, N, r = c["M"], c["K"], c["N"], c["r"]
    used = _touched(c["L"], 0.9 if c["mixed"] else 1.0, M)
    rank = 0.625 * r if c["mixed"] else r           # ranks are r, r/2 or r/4 where mixed
    live = 0.9 * M if c["mixed"] else M             # tokens with an adapter
    nb = used * rank * (K + N) * 2 + 4 * M
    fl = 2.0 * live * rank * (K + N)
    if c["fused"]:
        return {"bytes": nb + M * K * 2 + M * N * 2 + N * K * (0.5 + 2.5 / GROUP),
                "flops": fl + 2.0 * M * N * K}
    return {"bytes": nb + live * K * 2 + M * N * 4, "flops": fl}


# ----------------------------------------------------------------- prepare ---

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _activations(g, M, K):
    """N(0, 1) with 2 % outlier channels twenty times as large, as the
    activations of large models have them; bf16."""
    x = _randn(g, M, K)
    out = torch.rand(K, generator=g, device=DEV) < 0.02
    return (x * torch.where(out, 20.0, 1.0)).to(torch.bfloat16)


def _w4(g, *shape):
    """Codes, scales and zero points of packed int4 weights [..., N, K]: codes
    around a zero point near the middle of the grid."""
    groups = shape[:-1] + (shape[-1] // GROUP,)
    zero = torch.randint(5, 11, groups, generator=g, device=DEV, dtype=torch.uint8)
    q = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).mul_(3.0)
    q = q.view(*groups, GROUP).add_(zero[..., None]).round_().clamp_(0, 15)
    scale = (_randn(g, *groups).abs_() * (0.02 / 7.0) + 1e-4).to(torch.float16)
    return q.to(torch.uint8).view(shape), scale, zero


def _picks(g, T, E, k):
    """k different experts a token, some experts more popular than others, and
    positive weights that sum to one."""
    logits = _randn(g, T, E) + 0.5 * _randn(g, E)
    val, ids = torch.topk(logits, k, dim=1)
    w = torch.exp(val - val.max(dim=1, keepdim=True).values)
    return ids.to(torch.int32), (w / w.sum(dim=1, keepdim=True)).contiguous()


def _ranks(g, L, r, mixed):
    if not mixed:
        return torch.full((L,), r, dtype=torch.int32, device=DEV)
    shift = torch.randint(0, 4, (L,), generator=g, device=DEV, dtype=torch.int32)
    return torch.clamp(r >> torch.where(shift == 3, 0, shift), min=1).to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] == "route":
        s["logits"] = (2.0 * _randn(g, c["T"], c["E"])).to(
            torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        s["bias"] = 0.1 * _randn(g, c["E"]) if c["bias"] else None
        if own:
            import w4a8_quantized_gemm_gb300 as eg
            s["eg"] = eg
            s["out"] = (torch.empty(c["T"], c["k"], device=DEV),
                        torch.empty(c["T"], c["k"], dtype=torch.int32, device=DEV))
        return s
    if c["op"] == "experts":
        T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
        s["x"] = _activations(g, T, H)
        s["ids"], s["w"] = _picks(g, T, E, k)
        if c["dropped"]:
            drop = torch.rand(T, k, generator=g, device=DEV) < c["dropped"]
            s["ids"] = torch.where(drop, -1, s["ids"])
        gate_up = _w4(g, E, 2 * I, H)               # rows 0..I-1 gate, I..2I-1 up
        down = _w4(g, E, H, I)
        if own:
            import w4a8_quantized_gemm_gb300 as eg
            s["eg"] = eg
            s["layer"] = eg.moe_pack(*gate_up, *down)
            s["variant"] = eg.VARIANT_W4A8 if c["variant"] == "w4a8" else eg.VARIANT_W4A16
            s["ws"] = eg.moe_workspace(T, k, E, H, I, s["variant"], DEV)
            s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        else:
            s["gate_up"], s["down"] = gate_up, down
        return s
    M, L, r, K, N = c["M"], c["L"], c["r"], c["K"], c["N"]
    s["x"] = _activations(g, M, K)
    s["A"] = (_randn(g, L, r, K) / math.sqrt(K)).to(torch.bfloat16)
    s["B"] = (_randn(g, L, N, r) / math.sqrt(r)).to(torch.bfloat16)
    s["ranks"] = _ranks(g, L, r, c["mixed"])
    s["scale"] = torch.rand(L, generator=g, device=DEV) + 0.5
    ids = torch.randint(0, L, (M,), generator=g, device=DEV, dtype=torch.int32)
    if c["mixed"]:
        none = torch.rand(M, generator=g, device=DEV) < 0.1
        ids = torch.where(none, -1, ids)
    # requests of a batch lie side by side: in a prefill many rows of one
    s["ids"] = ids if M < 512 else torch.sort(ids).values
    if c["fused"]:
        s["weight"] = _w4(g, N, K)
    else:
        s["y"] = (3.0 * _randn(g, M, N)).to(torch.bfloat16)
    if own:
        import w4a8_quantized_gemm_gb300 as eg
        s["eg"] = eg
        s["adapters"] = eg.LoraAdapters(s["A"], s["B"], s["scale"], s["ranks"])
        s["out"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        if c["fused"]:
            s["packed"] = eg.pack_w4(*s.pop("weight"))
            s["ws"] = eg.w4a8_linear_lora_workspace(M, N, K, s["adapters"], DEV)
        else:
            s["ws"] = eg.lora_workspace(M, N, K, s["adapters"], DEV)
    return s


# --------------------------------------------------------------------- run ---

def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "experts": _own_experts, "lora": _own_lora}[op](state)
    return {"route": _plain_route, "experts": _plain_experts, "lora": _plain_lora}[op](state)


def _own_route(s):
    eg, c = s["eg"], s["case"]
    weights, ids = eg.moe_route(
        s["logits"], c["k"], bias=s["bias"],
        score=eg.SCORE_SIGMOID if c["score"] == "sigmoid" else eg.SCORE_SOFTMAX,
        n_group=c["groups"], topk_group=c["top_groups"],
        group_score=eg.GROUP_TOP2 if c["top2"] else eg.GROUP_MAX, renorm=c["renorm"],
        scale=c["scale"], out=s["out"])
    return {"weights": weights, "ids": ids}


def _own_experts(s):
    return s["eg"].moe_experts(s["x"], s["ids"], s["w"], s["layer"], variant=s["variant"],
                               workspace=s["ws"], out=s["out"])


def _own_lora(s):
    eg = s["eg"]
    if s["case"]["fused"]:
        return eg.w4a8_linear_lora(s["x"], s["packed"], s["case"]["N"], s["adapters"], s["ids"],
                                   workspace=s["ws"], out=s["out"])
    return eg.lora_add(s["y"], s["x"], s["adapters"], s["ids"], workspace=s["ws"], out=s["out"])


# ------------------------------------------------- the plain forms (32 bits) ---

def _first(v, n):
    """The n largest of each row, ties to the lowest index: values, indices."""
    val, idx = torch.sort(v, dim=-1, descending=True, stable=True)
    return val[..., :n], idx[..., :n]


def _plain_route(s):
    c = s["case"]
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    logits = s["logits"].float()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
        choice = score
    else:
        e = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
        score = e / e.sum(dim=1, keepdim=True)
        choice = logits                    # a softmax keeps the order of its logits
    if c["bias"]:
        choice = score + s["bias"]
    if c["top_groups"] < G:
        parts = choice.view(T, G, E // G)
        rank = _first(parts, 2)[0].sum(dim=-1) if c["top2"] else parts.max(dim=-1).values
        best = _first(rank, c["top_groups"])[1]
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, best, True)
        choice = torch.where(keep[..., None], parts, -math.inf).view(T, E)
    ids = _first(choice, k)[1]
    weights = torch.gather(score, 1, ids)
    if c["renorm"]:
        weights = weights / (weights.sum(dim=1, keepdim=True) + 1e-20)
    return {"weights": weights * c["scale"], "ids": ids.to(torch.int32)}


def _dequant(q, scale, zero):
    """fp32 weights [..., N, K]: scale * (code - zero)."""
    q = q.view(*q.shape[:-1], -1, GROUP).float()
    return ((q - zero.float()[..., None]) * scale.float()[..., None]).flatten(-2)


def _quantize(x):
    """Codes (as floats) and scales of each row: absmax / 127, to the nearest,
    ties to even."""
    a_s = x.float().abs().amax(dim=-1, keepdim=True) / 127.0
    a_q = torch.where(a_s > 0, x.float() / a_s, 0.0).round().clamp(-127, 127)
    return a_q, a_s


def _plain_experts(s):
    c = s["case"]
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
    flat = s["ids"].reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    key, slot = torch.sort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)
    start = torch.cumsum(counts, 0) - counts
    cap = max(1, int(counts[:E].max()))
    live = key < E
    key, slot = key[live], slot[live]
    rank = torch.arange(key.numel(), device=DEV) - start[key]
    rows = torch.zeros(E, cap, H, device=DEV)
    a8 = c["variant"] == "w4a8"
    x, x_s = _quantize(s["x"]) if a8 else (s["x"].float(), None)
    rows[key, rank] = x[slot // k]
    gu = torch.bmm(rows, _dequant(*s["gate_up"]).transpose(1, 2))
    if a8:
        sc = torch.zeros(E, cap, 1, device=DEV)
        sc[key, rank] = x_s[slot // k]
        gu = gu * sc
    gate, up = gu[..., :I], gu[..., I:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    if a8:
        # the int8 codes are those of bf16 activations, as for every W4A8 linear
        h, h_s = _quantize(h.to(torch.bfloat16))
    y = torch.bmm(h, _dequant(*s["down"]).transpose(1, 2))
    if a8:
        y = y * h_s
    parts = torch.zeros(T * k, H, device=DEV)
    parts[slot] = y[key, rank] * s["w"].reshape(-1)[slot][:, None]
    return parts.view(T, k, H).sum(dim=1).to(torch.bfloat16)


def _plain_lora(s):
    c = s["case"]
    M, L, r, N, K = c["M"], c["L"], c["r"], c["N"], c["K"]
    x, ids = s["x"].float(), s["ids"].long()
    at, live = torch.arange(M, device=DEV), (ids >= 0) & (ids < L)
    pick = torch.where(live, ids, 0)
    h = torch.mm(x, s["A"].float().view(L * r, K).t()).view(M, L, r)[at, pick]
    rank_ok = torch.arange(r, device=DEV)[None, :] < s["ranks"][pick][:, None]
    h = torch.where(rank_ok & live[:, None], h * s["scale"][pick][:, None], 0.0)
    wide = torch.zeros(M, L, r, device=DEV)
    wide[at, pick] = h
    delta = torch.mm(wide.view(M, L * r), s["B"].float().transpose(1, 2).reshape(L * r, N))
    if c["fused"]:
        a_q, a_s = _quantize(s["x"])
        y = torch.mm(a_q, _dequant(*s["weight"]).t()) * a_s
    else:
        y = s["y"].float()
    return (y + delta).to(torch.bfloat16)


# -------------------------------------------------- the definition in 64 bits ---

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"route": _exact_route, "experts": _exact_experts, "lora": _exact_lora}[case["op"]](s)


def _exact_route(s):
    c = s["case"]
    z = s["logits"].double()
    p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, dim=1)
    pick = p + s["bias"].double() if s["bias"] is not None else p
    T, per = c["T"], c["E"] // c["groups"]
    if c["groups"] > c["top_groups"]:
        by_group = pick.view(T, c["groups"], per)
        best = by_group.sort(dim=2, descending=True).values
        value = best[:, :, :2].sum(dim=2) if c["top2"] else best[:, :, 0]
        order = torch.argsort(value, dim=1, descending=True, stable=True)
        out = torch.ones_like(value, dtype=torch.bool)
        out.scatter_(1, order[:, :c["top_groups"]], False)
        pick = by_group.masked_fill(out[:, :, None], -math.inf).reshape(T, -1)
    ids = torch.argsort(pick, dim=1, descending=True, stable=True)[:, :c["k"]]
    w = torch.take_along_dim(p, ids, dim=1)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"weights": w * c["scale"], "ids": None}


def _codes(x):
    """The definition's int8 codes: an fp32 scale, the fp32 quotient rounded
    half to even (whole numbers, so they are the same in any precision)."""
    x = x.float()
    top = x.abs().max(dim=1).values
    a_s = torch.div(top, torch.full_like(top, 127.0))
    q = torch.round(torch.div(x, a_s[:, None]))
    q = torch.where((a_s == 0)[:, None], torch.zeros_like(q), q)
    return torch.clip(q, -127, 127).double(), a_s.double()


def _weights64(q, scale, zero):
    g = scale.shape[-1]
    d = q.double().view(-1, g, GROUP) - zero.double().view(-1, g, 1)
    return (d * scale.double().view(-1, g, 1)).view(q.shape)


def _exact_experts(s):
    c = s["case"]
    I, a8 = c["I"], c["variant"] == "w4a8"
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        tok, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if tok.numel() == 0:
            continue
        w1 = _weights64(*(t[e] for t in s["gate_up"]))
        w2 = _weights64(*(t[e] for t in s["down"]))
        if a8:
            q, a_s = _codes(s["x"][tok])
            gu = (q @ w1.t()) * a_s[:, None]
        else:
            gu = s["x"][tok].double() @ w1.t()
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        if a8:
            q, a_s = _codes(h.to(torch.bfloat16))
            y = (q @ w2.t()) * a_s[:, None]
        else:
            y = h @ w2.t()
        out.index_add_(0, tok, y * s["w"][tok, j].double()[:, None])
    return out


def _exact_lora(s):
    c = s["case"]
    if c["fused"]:
        q, a_s = _codes(s["x"])
        y = (q @ _weights64(*s["weight"]).t()) * a_s[:, None]
    else:
        y = s["y"].double()
    for a in range(c["L"]):
        rows = torch.nonzero(s["ids"] == a)[:, 0]
        if rows.numel() == 0:
            continue
        n = int(s["ranks"][a])
        h = s["x"][rows].double() @ s["A"][a, :n].double().t()
        d = h @ s["B"][a, :, :n].double().t()
        y[rows] += d * s["scale"][a].double()
    return y
