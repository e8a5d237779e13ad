"""The microscaled 4-bit linears, as work to be measured.

Two formats of e2m1 values {0, .5, 1, 1.5, 2, 3, 4, 6}: blocks of 32 with a power
of two for a scale ("e8m0"), and blocks of 16 with an e4m3 scale under one fp32
scale for the tensor ("e4m3"). Four operators:

  quant    rows to 4 bits and back to the values those stand for
  linear   rows to 4 bits, times a packed 4-bit weight
  ragged   the same over rows sorted by expert, each with its expert's weight;
           rows are gathered from the tokens on the way
  gated    silu(gate) * up of the gate and up halves to 4 bits, times the packed
           down weight (of one linear, or ragged)

`listed()` holds the cases, `draw(rng)` more of the same ranges, `prepare` makes
what a program has in hand, `run` is one pass. With `own` false a pass is the
operator's plain form in elementary torch operations in 32 bits (64 for the gated
values, which lie next to borders between codes); with `own` true it is the call
a user makes. `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = {"e8m0": 32, "e4m3": 16}
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one token's activations: latency only
        dict(name="quant-1", op="quant", fmt="e8m0", x="bf16", M=1, K=3584),
        # the widest activations of the largest prefill batch, ragged, fp16
        dict(name="quant-4093", op="quant", fmt="e4m3", x="f16", M=4093, K=18944),
        # one token through the gate or up projection: every weight byte once
        dict(name="linear-1", op="linear", fmt="e8m0", x="bf16", M=1, K=3584, N=18944),
        # a decode batch through q, k and v
        dict(name="linear-16", op="linear", fmt="e4m3", x="bf16", M=16, K=3584, N=4608),
        # logits of a few dozen sequences over an odd vocabulary, fp16
        dict(name="linear-77", op="linear", fmt="e4m3", x="f16", M=77, K=2048, N=50257),
        # the largest prefill batch through the gate or up projection
        dict(name="linear-4096", op="linear", fmt="e8m0", x="bf16", M=4096, K=3584, N=18944),
        # one token through its experts' gate and up projections
        dict(name="ragged-1", op="ragged", fmt="e8m0", x="bf16", T=1, E=64, k=8, K=3584, N=2560,
             dropped=0.0),
        # a decode batch: a few rows an expert
        dict(name="ragged-33", op="ragged", fmt="e4m3", x="bf16", T=33, E=64, k=8, K=3584, N=2560,
             dropped=0.0),
        # the largest prefill batch through the experts' gate and up projections
        dict(name="ragged-4096", op="ragged", fmt="e8m0", x="bf16", T=4096, E=64, k=8, K=3584,
             N=2560, dropped=0.0),
        # one token through the down projection
        dict(name="gated-1", op="gated", fmt="e8m0", x="bf16", M=1, K=18944, N=3584),
        # a ragged prefill chunk through the down projection
        dict(name="gated-1021", op="gated", fmt="e4m3", x="bf16", M=1021, K=18944, N=3584),
        # a ragged prefill batch through the experts' down projections; a quarter
        # of the picks belong to experts of another machine
        dict(name="gated-ragged-2977", op="gated", fmt="e4m3", x="bf16", T=2977, E=64, k=6, K=1408,
             N=2048, dropped=0.25),
    ]


def draw(rng):
    """One more case of the ranges above (no name)."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quant", "linear", "ragged", "gated"])
    c = dict(op=op, fmt=rng.choice(["e8m0", "e4m3"]), x=rng.choice(["bf16", "bf16", "f16"]))
    if op == "quant":
        return dict(c, M=log_int(1, 4093), K=32 * log_int(4, 592))
    if op == "ragged" or (op == "gated" and rng.random() < 0.4):
        E = rng.choice([8, 16, 24, 32, 48, 64])
        T, k = log_int(1, 4096), rng.randint(1, 8)
        return dict(c, T=T, E=E, k=k, K=32 * rng.randint(8, 112 if op == "ragged" else 44),
                    N=rng.choice([1, 8, 64]) * rng.randint(4, 40),
                    dropped=0.25 if T * k >= 16 and rng.random() < 0.5 else 0.0)
    K = 32 * log_int(8, 112 if op == "linear" else 592)
    return dict(c, M=log_int(1, 4096), K=K, N=log_int(128, min(50257, 2 ** 26 // K)))


# -------------------------------------------------------------------- work ---

def work(case):
    c = case
    K, size = c["K"], 4 if c["x"] == "f32" else 2
    held = 0.5 + 1.0 / BLOCK[c["fmt"]]              # bytes of a value in 4 bits
    if c["op"] == "quant":
        return {"bytes": c["M"] * K * (2 * size + 2 * held), "flops": 4.0 * c["M"] * K}
    halves = 2 if c["op"] == "gated" else 1
    if "T" not in c:
        M, N = c["M"], c["N"]
        return {"bytes": M * K * halves * size + N * K * held + M * N * size,
                "flops": 2.0 * M * N * K}
    T, E, k, N = c["T"], c["E"], c["k"], c["N"]
    live = 1.0 - c["dropped"]
    rows = T * k * live
    touched = E * (1.0 - (1.0 - k * live / E) ** T)
    read = T * K if c["op"] == "ragged" else 2 * rows * K
    return {"bytes": read * size + touched * N * K * held + rows * N * size + 4 * (T * k + E),
            "flops": 2.0 * rows * N * K}


# ----------------------------------------------------------------- prepare ---

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _activations(g, M, K, dtype):
    """N(0, 1) with 2 % outlier channels twenty times as large, as the
    activations of large models have them."""
    x = _randn(g, M, K)
    out = torch.rand(K, generator=g, device=DEV) < 0.02
    return (x * torch.where(out, 20.0, 1.0)).to(dtype)


def _tensor_scale(fmt, top):
    """The fp32 scale that brings the largest block's e4m3 scale to its top."""
    return (top.float() / (6.0 * 448.0)).reshape(-1) if fmt == "e4m3" else None


def _weight(g, fmt, *shape):
    """A checkpoint's 4-bit weight [..., N, K]: codes, two to a byte, block
    scales, and the tensors' scales [...]."""
    w = _randn(g, *shape) * 0.02
    ts = _tensor_scale(fmt, w.abs().amax(dim=(-2, -1)))
    mag, neg, _, byte = _split(w if ts is None else w * (1.0 / ts).view(-1, 1, 1).view(
        *shape[:-2], 1, 1), fmt)
    code = (mag + 8 * neg.to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte, ts


def _sorted_picks(g, c):
    """k different experts a token, some more popular than others, and the picks
    sorted by expert: the token of each sorted row, and each expert's first row."""
    T, E, k = c["T"], c["E"], c["k"]
    ids = torch.topk(_randn(g, T, E) + 0.5 * _randn(g, E), k, dim=1).indices.reshape(-1)
    if c["dropped"]:
        ids = torch.where(torch.rand(T * k, generator=g, device=DEV) < c["dropped"], E, ids)
    ids, order = torch.sort(ids, stable=True)
    first = torch.searchsorted(ids, torch.arange(E + 1, device=DEV))
    return (order // k).to(torch.int32), first.to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 31)
    fmt, K, dtype = c["fmt"], c["K"], DTYPE[c["x"]]
    s = dict(case=c)
    ragged, gated = "T" in c, c["op"] == "gated"
    n = c["T"] * c["k"] if ragged else c["M"]
    if ragged:
        s["index"], s["offsets"] = _sorted_picks(g, c)
    if gated:
        # the gate and up projections' output of each row
        s["index"] = None
        s["x"] = (1.5 * _randn(g, n, 2 * K)).to(dtype)
        # (calibrated, with room: the largest of a batch is seldom larger)
        top = torch.full((1,), 24.0, device=DEV)
    else:
        s["x"] = _activations(g, c["T"] if ragged else n, K, dtype)
        top = s["x"].abs().max()
    s["ts"] = _tensor_scale(fmt, top)
    if c["op"] != "quant":
        N = c["N"]
        s["weight"] = _weight(g, fmt, *((c["E"], N, K) if ragged else (N, K)))
        # (rows of no expert keep what they held)
        s["out"] = torch.zeros(n, N, dtype=dtype, device=DEV)
    if own:
        import w4a8_quantized_gemm_gb300 as eg
        s["eg"] = eg
        s["fmt"] = eg.MX4_E8M0 if fmt == "e8m0" else eg.MX4_E4M3
        if c["op"] == "quant":
            s["out"] = torch.empty(n, K, dtype=dtype, device=DEV)
        else:
            code, scale, ts = s.pop("weight")
            s["weight"] = eg.mx4_pack(code, scale, s["fmt"], tensor_scale=ts)
            s["ws"] = eg.mx4_workspace(n, s["weight"], DEV)
    return s


# --------------------------------------------------------------------- run ---

def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    if c["op"] == "quant":
        v = _plain_rows(s, c)
        return (v if s["ts"] is None else v * s["ts"]).to(s["x"].dtype)
    if "T" in c:
        return _plain_ragged(s, c)
    return _plain_linear(s, c)


def _own(s, c):
    eg = s["eg"]
    if c["op"] == "quant":
        rows = eg.mx4_quant(s["x"], s["fmt"], tensor_scale=s["ts"], with_tc=False)
        return eg.mx4_dequant(rows, dtype=s["x"].dtype, out=s["out"])
    gated = c["op"] == "gated"
    if "T" in c:
        return eg.mx4_linear_ragged(s["x"], s["offsets"], s["weight"], index=s["index"],
                                    tensor_scale=s["ts"], gated=gated, out=s["out"],
                                    workspace=s["ws"])
    return eg.mx4_linear(s["x"], s["weight"], tensor_scale=s["ts"], gated=gated, out=s["out"],
                         workspace=s["ws"])


# ------------------------------------------------- the plain forms (32 bits) ---

def _power(e):
    """2^e in fp32 for whole e in [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _e4m3(v):
    """The e4m3 numbers nearest to v >= 0, ties to even, at most 448."""
    step = _power(torch.clamp(torch.frexp(v).exponent - 1, min=-6) - 3)
    return torch.clamp(torch.round(v / step) * step, max=448.0).float()


def _magnitude(v):
    """Codes 0..7 of the e2m1 magnitudes nearest to v >= 0, ties to even codes."""
    return ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5)
            + (v >= 3.5) + (v > 5.0))


def _split(x, fmt):
    """Blocks of x (over the tensor's scale): magnitudes' codes, signs, the blocks'
    scales in fp32 and as bytes."""
    u = x.unflatten(-1, (-1, BLOCK[fmt]))
    top = u.abs().amax(dim=-1, keepdim=True)
    if fmt == "e4m3":
        # (divided by a tensor: a division by a number is a product with its
        # rounded reciprocal, which is off next to a border)
        scale = _e4m3(top / torch.full_like(top, 6.0))
        byte = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
        scale, byte = _power(e), (e + 127).to(torch.uint8)
    mag = _magnitude(torch.where(scale > 0, u.abs() / scale, 0.0))
    return mag, u < 0, scale, byte.squeeze(-1)


def _value(mag):
    m = mag.float()
    return torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))


def _plain_values(x, fmt):
    """The values that x's codes stand for."""
    mag, neg, scale, _ = _split(x, fmt)
    return (_value(mag) * torch.where(neg, -scale, scale)).flatten(-2)


def _plain_rows(s, c):
    """The rows' values, over the tensor's scale."""
    x, ts = s["x"], s["ts"]
    if c["op"] != "gated":
        return _plain_values(x.float() if ts is None else x.float() * (1.0 / ts), c["fmt"])
    gate, up = x[..., :c["K"]].double(), x[..., c["K"]:].double()
    h = gate / (1.0 + torch.exp(-gate)) * up
    return _plain_values(h if ts is None else h * (1.0 / ts).double(), c["fmt"])


def _plain_weight(weight, fmt):
    """The weight's values in fp32, over the tensors' scales."""
    packed, scale, _ = weight
    code = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)
    v = _value(code & 7)
    v = torch.where(code >= 8, -v, v).unflatten(-1, (-1, BLOCK[fmt]))
    if fmt == "e8m0":
        sc = _power(scale.int() - 127)
    else:
        sc = scale.view(torch.float8_e4m3fn).float()
    return (v * sc[..., None]).flatten(-2)


def _plain_linear(s, c):
    y = torch.mm(_plain_rows(s, c), _plain_weight(s["weight"], c["fmt"]).t())
    if s["ts"] is not None:
        y = y * (s["ts"] * s["weight"][2])
    return s["out"].copy_(y.to(s["x"].dtype))


def _plain_ragged(s, c):
    E, K = c["E"], c["K"]
    rows, first = _plain_rows(s, c), s["offsets"].long()
    counts = first[1:] - first[:-1]
    cap, live = max(1, int(counts.max())), int(first[-1])
    at = torch.arange(live, device=DEV)
    e = torch.searchsorted(first[1:].contiguous(), at, right=True)
    wide = torch.zeros(E, cap, K, device=DEV)
    wide[e, at - first[e]] = rows[:live] if s["index"] is None else rows[s["index"][:live].long()]
    y = torch.bmm(wide, _plain_weight(s["weight"], c["fmt"]).transpose(1, 2))
    if s["ts"] is not None:
        y = y * (s["ts"] * s["weight"][2])[:, None, None]
    s["out"][:live] = y[e, at - first[e]].to(s["x"].dtype)
    return s["out"]


# -------------------------------------------------- the definition in 64 bits ---

def _pow64(e):
    """2^e in 64 bits, exactly (a power function is off by a last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round64(v, bits, lowest):
    """v >= 0 to numbers of `bits` bits whose smallest power of two is 2^lowest,
    ties to even, in 64 bits."""
    e = torch.floor(torch.log2(torch.clamp(v, min=2.0 ** lowest)))
    e = torch.where(_pow64(e) > v, e - 1, e).clamp(min=lowest)
    unit = _pow64(e - (bits - 1))
    return torch.round(v / unit) * unit


def _values64(x, fmt, ts):
    """The values that 4 bits hold of x: real numbers times the rounded
    reciprocal of the tensor's scale, if there is one, rounded once to fp32
    where x is a stored number (the gated values never are)."""
    stored = x.dtype is not torch.float64
    u = x.double()
    if ts is not None:
        u = u * torch.reciprocal(ts).double()
        u = u.float().double() if stored else u
    b = u.reshape(*u.shape[:-1], -1, BLOCK[fmt])
    top = b.abs().max(dim=-1, keepdim=True).values
    if fmt == "e8m0":
        e = torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -149)))
        e = torch.where(_pow64(e) > top, e - 1, torch.where(
            _pow64(e + 1) <= top, e + 1, e))
        scale = _pow64(torch.clamp(e - 2, -127, 127))
    else:
        scale = torch.clamp(_round64(top / torch.full_like(top, 6.0), 4, -6), max=448.0)
    q = torch.clamp(_round64(b.abs() / torch.where(scale == 0, 1.0, scale), 2, 0), max=6.0)
    return (torch.sign(b) * q * scale).reshape(u.shape)


def _weight64(weight, fmt):
    packed, scale, _ = weight
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float64, device=DEV)
    v = torch.empty(*packed.shape[:-1], packed.shape[-1], 2, dtype=torch.float64, device=DEV)
    v[..., 0], v[..., 1] = table[(packed % 16).long()], table[(packed // 16).long()]
    if fmt == "e8m0":
        sc = _pow64(scale.double() - 127.0)
    else:
        sc = scale.view(torch.float8_e4m3fn).double()
    return v.reshape(*sc.shape, -1).mul_(sc[..., None]).reshape(*packed.shape[:-1], -1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, fmt, ts = case, case["fmt"], s["ts"]
    x = s["x"]
    if c["op"] == "gated":
        gate, up = x.double().split(c["K"], dim=1)
        x = torch.nn.functional.silu(gate) * up
    rows = _values64(x, fmt, ts)
    g = 1.0 if ts is None else ts.double()
    if c["op"] == "quant":
        return rows * g
    codes, scale, wts = s["weight"]
    wg = None if wts is None else wts.double()
    if "T" not in c:
        y = rows @ _weight64(s["weight"], fmt).t()
        return y if wg is None else y * (g * wg)
    if s["index"] is not None:
        rows = rows[s["index"].long()]
    y = torch.zeros(rows.shape[0], c["N"], dtype=torch.float64, device=DEV)
    first = s["offsets"].tolist()
    for e in range(c["E"]):
        a, b = first[e], first[e + 1]
        if a < b:
            w = _weight64((codes[e], scale[e], None), fmt)
            y[a:b] = (rows[a:b] @ w.t()) * (1.0 if wg is None else g * wg[e])
    return y
