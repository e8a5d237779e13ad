"""GPU tests of the operators whose weights each row picks: the router, the
experts' gated linears, the low-rank adapters -- each against a plain
implementation in 64 bits.

Tolerances, derived from the roundings a result passes through (u = 2^-8, half
a bf16 spacing relative to the value: eight significant bits):
- router weights: fp32, a few roundings of 2^-24 and expf's 2 ulp: 1e-5;
- adapters: y = bf16(y0 + B bf16(s A x)): u |y| + u sum |B| |s A x|, and the
  fp32 sums' 2^-18 of sum |B| s sum |A| |x| (K below 2^13 terms);
- experts: bf16(sum_j w_j bf16(D_j bf16(h_j))): u |out| + u sum w |y_j| +
  u sum w |D_j| |h_j|, and 2^-14 of the last sum for the fp32 sums and the fast
  exponential behind h. W4A8 quantizes bf16(h): where the fp32 sums move h over
  a bf16 boundary its code can move by one, so a few codes' worth, each h_s |D|,
  comes on top. All three roundings are independent, so the whole result is
  within 4e-3 in the 2-norm (a rounding's root mean square is about 0.42 u: three
  of them 2.8e-3).
"""
import math

import numpy as np
import pytest
import torch

import w4a8_quantized_gemm_gb300 as eg

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------- router ---

def route_ref(logits, k, bias, score, n_group, topk_group, group_score, renorm, scale):
    """(weights, choice [T, E] with -inf outside the kept groups), fp64."""
    z = logits.double()
    z = torch.where(torch.isnan(z), -math.inf, z).clamp(max=3.402823466e38)
    if score == eg.SCORE_SIGMOID:
        s = torch.sigmoid(z)
    else:
        m = z.max(dim=1, keepdim=True).values
        e = torch.exp(z - torch.where(torch.isinf(m), 0.0, m))
        s = e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)
    c = s + bias.double() if bias is not None else s
    T, E = c.shape
    if topk_group < n_group:
        part = c.view(T, n_group, E // n_group)
        n2 = min(2, E // n_group) if group_score == eg.GROUP_TOP2 else 1
        v = part.topk(n2, dim=2).values.sum(dim=2)
        order = torch.argsort(v, dim=1, descending=True, stable=True)[:, :topk_group]
        keep = torch.zeros_like(v, dtype=torch.bool).scatter_(1, order, True)
        c = part.masked_fill(~keep[:, :, None], -math.inf).reshape(T, E)
    return s, c


def check_route(logits, k, **kw):
    kw = dict(dict(bias=None, score=eg.SCORE_SOFTMAX, n_group=1, topk_group=1,
                   group_score=eg.GROUP_MAX, renorm=True, scale=1.0), **kw)
    w, ids = eg.moe_route(logits, k, **kw)
    s, c = route_ref(logits, k, **kw)
    T, E = c.shape
    assert ids.min() >= 0 and ids.max() < E
    picked = torch.gather(c, 1, ids.long())
    for j in range(k):
        for i in range(j):
            assert not (ids[:, i] == ids[:, j]).any(), "an expert was picked twice"
    # the picks are the largest choices, in order, up to the fp32 arithmetic
    best = c.sort(dim=1, descending=True).values[:, :k]
    assert torch.equal(torch.isinf(picked), torch.isinf(best))
    f = torch.isfinite(best)
    assert (picked - best)[f].abs().max().item() <= 2e-6 if f.any() else True
    ref = torch.gather(s, 1, ids.long())
    if kw["renorm"]:
        ref = ref / (ref.sum(dim=1, keepdim=True) + 1e-20)
    ref = ref * kw["scale"]
    assert torch.allclose(w.double(), ref, rtol=1e-5, atol=1e-30)
    return w, ids


@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 1, 1, torch.float32), (1, 8, 8, torch.bfloat16), (3, 33, 4, torch.float32),
    (130, 64, 6, torch.bfloat16), (77, 160, 7, torch.float32), (5, 512, 32, torch.float32),
    (1000, 257, 8, torch.bfloat16)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_plain(T, E, k, dtype, score):
    x = (2 * torch.randn(T, E, generator=gen(T + E), device=DEV)).to(dtype)
    check_route(x, k, score=score, renorm=bool(T % 2), scale=1.0 if T % 2 else 2.5)


@pytest.mark.parametrize("E,groups,keep,k", [
    (256, 8, 4, 8), (64, 8, 1, 8), (160, 8, 3, 6), (32, 32, 5, 5), (24, 4, 3, 4), (512, 2, 1, 9)])
@pytest.mark.parametrize("score,top2,bias", [(0, 0, False), (1, 1, True), (0, 1, True),
                                             (1, 0, False), (0, 1, False)])
def test_route_groups(E, groups, keep, k, score, top2, bias):
    g = gen(E + keep)
    x = 2 * torch.randn(201, E, generator=g, device=DEV)
    b = 0.1 * torch.randn(E, generator=g, device=DEV) if bias else None
    check_route(x, k, score=score, n_group=groups, topk_group=keep, group_score=top2, bias=b)


def test_route_ties_go_to_the_lowest_index():
    x = torch.zeros(9, 96, device=DEV)
    w, ids = check_route(x, 5)
    assert torch.equal(ids, torch.arange(5, dtype=torch.int32, device=DEV).expand(9, 5))
    w, ids = check_route(x, 4, n_group=8, topk_group=2, group_score=eg.GROUP_TOP2,
                         score=eg.SCORE_SIGMOID)
    assert torch.equal(ids, torch.arange(4, dtype=torch.int32, device=DEV).expand(9, 4))
    x[:, 40] = x[:, 90] = 1.0
    w, ids = check_route(x, 3, score=eg.SCORE_SIGMOID)
    assert ids[0].tolist() == [40, 90, 0]
    # zeros of either sign tie
    x = torch.zeros(2, 40, device=DEV)
    x[:, :3] = -0.0
    assert eg.moe_route(x, 3)[1][0].tolist() == [0, 1, 2]


def test_route_masked_and_non_finite_logits():
    inf, nan = math.inf, math.nan
    x = torch.randn(6, 64, device=DEV)
    x[0] = -inf                      # every expert masked off: scores of zero
    x[1, 3:] = -inf                  # three left, four picked
    x[2, 5] = nan
    x[3, 7] = inf
    x[4] = torch.finfo(torch.float32).min
    for score in (eg.SCORE_SOFTMAX, eg.SCORE_SIGMOID):
        w, ids = eg.moe_route(x, 4, score=score)
        assert torch.isfinite(w).all()
        assert ids[0].tolist() == [0, 1, 2, 3] and w[0].abs().max() == 0
        assert sorted(ids[1, :3].tolist()) == [0, 1, 2] and w[1, 3] == 0
        assert 5 not in ids[2].tolist()
        assert ids[3, 0] == 7
        if score == eg.SCORE_SOFTMAX:
            assert w[3, 0] == 1.0
            assert torch.allclose(w[4], torch.full((4,), 0.25, device=DEV))
        check_route(x[1:2], 3, score=score)


# ------------------------------------------------------------------ experts ---

def w4(g, *shape):
    groups = shape[:-1] + (shape[-1] // 128,)
    return (torch.randint(0, 16, shape, generator=g, device=DEV, dtype=torch.uint8),
            (torch.randn(groups, generator=g, device=DEV).abs() * 0.003 + 1e-4).half(),
            torch.randint(0, 16, groups, generator=g, device=DEV, dtype=torch.uint8))


def dequant64(q, s, z):
    q = q.double().view(*q.shape[:-1], -1, 128)
    return ((q - z.double()[..., None]) * s.double()[..., None]).flatten(-2)


def codes64(x):
    a_s = x.float().abs().amax(dim=1) / 127.0
    q = (x.float() / a_s[:, None]).round().clamp(-127, 127)
    q = torch.where(a_s[:, None] > 0, q, 0.0)
    return q.double(), a_s.double()


def experts_case(seed, T, E, k, H, I):
    g = gen(seed)
    x = torch.randn(T, H, generator=g, device=DEV)
    x[:, ::50] *= 20.0
    scores = torch.randn(T, E, generator=g, device=DEV)
    w, ids = torch.topk(scores, k, dim=1)
    return (x.bfloat16(), ids.int(), torch.softmax(w, dim=1).contiguous(), w4(g, E, 2 * I, H),
            w4(g, E, H, I))


def experts_ref(x, ids, w, gate_up, down, variant):
    T, H = x.shape
    E, I2, _ = gate_up[0].shape
    I = I2 // 2
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(out)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        w1 = dequant64(*(v[e] for v in gate_up))
        w2 = dequant64(*(v[e] for v in down))
        if variant == eg.VARIANT_W4A8:
            q, a_s = codes64(x[t])
            gu = (q @ w1.T) * a_s[:, None]
        else:
            gu = x[t].double() @ w1.T
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        if variant == eg.VARIANT_W4A8:
            q, h_s = codes64(h.bfloat16())
            h = q * h_s[:, None]
            more = 4 * h_s[:, None] * w2.abs().max()
        else:
            more = 0.0
        y = h @ w2.T
        wt = w[t, j].double()[:, None]
        out.index_add_(0, t, wt * y)
        bound.index_add_(0, t, wt.abs() * (1.1 * U * y.abs() + (U + 2.0 ** -14) *
                                           (h.abs() @ w2.abs().T) + more))
    return out, bound + U * out.abs() + 1e-30


def check_experts(case, variant, path, **kw):
    x, ids, w, gate_up, down = case
    layer = eg.moe_pack(*gate_up, *down)
    y = eg.moe_experts(x, ids, w, layer, variant=variant, path=path, **kw)
    ref, bound = experts_ref(x, ids, w, gate_up, down, variant)
    err = (y.double() - ref).abs()
    assert torch.isfinite(y.float()).all()
    assert (err <= bound).all(), (err / bound).max().item()
    norm = ref.norm().item()
    assert err.norm().item() <= 4e-3 * norm + 1e-30, err.norm().item() / norm
    assert eg.device_status() == 0
    return y


VARIANTS = [eg.VARIANT_W4A16, eg.VARIANT_W4A8]


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 8, 2, 256, 128), (1, 1, 1, 128, 128), (2, 3, 3, 384, 256), (7, 64, 6, 512, 128),
    (8, 16, 4, 128, 384), (9, 4, 2, 1152, 256), (17, 5, 5, 256, 1152), (33, 8, 3, 640, 128),
    (65, 2, 2, 256, 256), (300, 7, 3, 384, 256)])
def test_experts_stream(variant, T, E, k, H, I):
    check_experts(experts_case(T + E, T, E, k, H, I), variant, eg.PATH_GEMV)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 128, 128), (3, 4, 2, 256, 128), (40, 3, 2, 384, 256), (191, 1, 1, 256, 128),
    (192, 2, 2, 128, 256), (193, 2, 1, 256, 256), (500, 6, 3, 640, 384), (333, 40, 4, 256, 128),
    (1500, 5, 2, 256, 1152), (700, 200, 8, 128, 128)])
def test_experts_tensor_cores(variant, T, E, k, H, I):
    check_experts(experts_case(T + E, T, E, k, H, I), variant, eg.PATH_TC)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("path", [eg.PATH_GEMV, eg.PATH_TC])
def test_experts_dropped_repeated_and_skewed_picks(variant, path):
    x, ids, w, gu, dn = experts_case(5, 70, 6, 3, 256, 128)
    ids[::3] = -1                              # tokens without any expert
    ids[1::3, 1] = 6                           # beyond the last one
    ids[2::3, 0] = -2 ** 31
    y = check_experts((x, ids, w, gu, dn), variant, path)
    assert (y[::3] == 0).all()
    ids = torch.full_like(ids, -1)             # nothing at all
    layer = eg.moe_pack(*gu, *dn)
    assert (eg.moe_experts(x, ids, w, layer, variant=variant, path=path) == 0).all()
    ids = torch.full_like(ids, 4)              # one expert takes every pick
    check_experts((x, ids, w, gu, dn), variant, path)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("path", [eg.PATH_GEMV, eg.PATH_TC])
def test_experts_zero_rows_weights_and_empty_batch(variant, path):
    x, ids, w, gu, dn = experts_case(6, 20, 4, 2, 256, 128)
    x[3] = 0
    w[5] = 0
    layer = eg.moe_pack(*gu, *dn)
    y = eg.moe_experts(x, ids, w, layer, variant=variant, path=path)
    assert (y[3] == 0).all() and (y[5] == 0).all()
    check_experts((x, ids, w, gu, dn), variant, path)
    assert eg.moe_experts(x[:0], ids[:0], w[:0], layer, variant=variant).shape == (0, 256)


@pytest.mark.parametrize("path", [eg.PATH_GEMV, eg.PATH_TC])
def test_experts_on_another_stream_and_again_in_one_workspace(path):
    case = experts_case(7, 40, 8, 4, 384, 256)
    x, ids, w, gu, dn = case
    layer = eg.moe_pack(*gu, *dn)
    ws = eg.moe_workspace(40, 4, 8, 384, 256, eg.VARIANT_W4A8, DEV, path)
    ws.fill_(0xFF)                             # NaN patterns: nothing stale is read
    want = check_experts(case, eg.VARIANT_W4A8, path, workspace=ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    outs = [eg.moe_experts(x, ids, w, layer, workspace=ws, path=path, stream=st)
            for _ in range(3)]
    few = eg.moe_experts(x[:3], ids[:3].contiguous(), w[:3].contiguous(), layer, workspace=ws,
                         path=path, stream=st)
    st.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    ref, bound = experts_ref(x[:3], ids[:3], w[:3], gu, dn, eg.VARIANT_W4A8)
    assert ((few.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("T,path", [(6, eg.PATH_GEMV), (90, eg.PATH_GEMV), (90, eg.PATH_TC),
                                    (700, eg.PATH_TC)])
def test_experts_non_finite_rows_stay_alone(variant, T, path):
    x, ids, w, gu, dn = experts_case(11, T, 4, 2, 256, 128)
    layer = eg.moe_pack(*gu, *dn)
    clean = eg.moe_experts(x, ids, w, layer, variant=variant, path=path)
    x[2, 5] = math.nan
    x[4, 200] = math.inf
    y = eg.moe_experts(x, ids, w, layer, variant=variant, path=path)
    other = torch.ones(T, dtype=torch.bool, device=DEV)
    other[[2, 4]] = False
    assert torch.equal(y[other], clean[other])
    if variant == eg.VARIANT_W4A16:
        assert not torch.isfinite(y[2].float()).any() and not torch.isfinite(y[4].float()).all()
    assert eg.device_status() == 0


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("T,path", [(5, eg.PATH_GEMV), (60, eg.PATH_GEMV), (60, eg.PATH_TC),
                                    (500, eg.PATH_TC)])
@pytest.mark.parametrize("low,high", [(-24, -14), (-20, 2), (0, 12)])
def test_experts_scales_of_the_whole_range(variant, T, path, low, high):
    """fp16 scales of 2^low to 2^high, subnormal ones among them."""
    x, ids, w, gu, dn = experts_case(12, T, 4, 2, 384, 256)
    g = gen(13)

    def spread(v):
        e = torch.randint(low, high, v[1].shape, generator=g, device=DEV)
        m = 1 + torch.rand(v[1].shape, generator=g, device=DEV) * 0.99
        return v[0], torch.ldexp(m, e).half(), v[2]

    check_experts((x, ids, w, spread(gu), spread(dn)), variant, path)


def test_gate_up_packing_interleaves_rows():
    g = gen(9)
    E, I, H = 3, 256, 256
    gu, dn = w4(g, E, 2 * I, H), w4(g, E, H, I)
    layer = eg.moe_pack(*gu, *dn)
    q, s, z = eg.unpack_w4(layer.gate_up, E * 2 * I, H)
    n = np.arange(2 * I)
    src = torch.from_numpy((n % 32 // 16) * I + n // 32 * 16 + n % 16).to(DEV)
    assert torch.equal(q.view(E, 2 * I, H), gu[0][:, src])
    assert torch.equal(s.view(E, 2 * I, -1), gu[1][:, src])
    assert torch.equal(z.view(E, 2 * I, -1), gu[2][:, src])
    q, s, z = eg.unpack_w4(layer.down, E * H, I)
    assert torch.equal(q.view(E, H, I), dn[0])


# ----------------------------------------------------------------- adapters ---

def lora_case(seed, M, N, K, L, r, mixed):
    g = gen(seed)
    x = torch.randn(M, K, generator=g, device=DEV)
    x[:, ::64] *= 20.0
    A = (torch.randn(L, r, K, generator=g, device=DEV) / math.sqrt(K)).bfloat16()
    B = torch.randn(L, N, r, generator=g, device=DEV).bfloat16()
    scale = torch.rand(L, generator=g, device=DEV) + 0.5
    ids = torch.randint(-1 if mixed else 0, L, (M,), generator=g, device=DEV, dtype=torch.int32)
    ranks = torch.randint(0, r + 1, (L,), generator=g, device=DEV,
                          dtype=torch.int32) if mixed else None
    y = torch.randn(M, N, generator=g, device=DEV).bfloat16()
    return y, x.bfloat16(), eg.LoraAdapters(A, B, scale, ranks), ids


def lora_ref(y, x, ad, ids):
    out = y.double().clone()
    bound = torch.zeros_like(out)
    for a in range(ad.L):
        rows = torch.nonzero(ids == a)[:, 0]
        n = ad.r if ad.ranks is None else max(0, min(ad.r, int(ad.ranks[a])))
        if rows.numel() == 0 or n == 0:
            continue
        s = ad.scale[a].double()
        Aa, Ba = ad.A[a, :n].double(), ad.B[a, :, :n].double()
        h = s * (x[rows].double() @ Aa.T)
        ha = s.abs() * (x[rows].double().abs() @ Aa.abs().T)
        out[rows] += h @ Ba.T
        bound[rows] = 1.01 * U * (h.abs() @ Ba.abs().T) + 2.0 ** -18 * (ha @ Ba.abs().T)
    return out, bound + 1.01 * U * out.abs() + 1e-30


def check_lora(y, x, ad, ids, **kw):
    got = eg.lora_add(y, x, ad, ids, **kw)
    ref, bound = lora_ref(y, x, ad, ids)
    err = (got.double() - ref).abs()
    assert (err <= bound).all(), (err / bound).max().item()
    none = (ids < 0) | (ids >= ad.L)
    assert torch.equal(got[none], y[none])
    return got


@pytest.mark.parametrize("M,N,K,L,r,mixed", [
    (1, 128, 128, 1, 8, False), (1, 3584, 3584, 32, 16, False), (2, 256, 384, 5, 24, True),
    (16, 384, 256, 1, 32, False), (17, 128, 1152, 3, 64, True), (67, 640, 512, 64, 32, True),
    (129, 256, 256, 40, 128, True), (500, 384, 640, 2, 16, True), (1025, 128, 256, 9, 72, True)])
def test_lora_add(M, N, K, L, r, mixed):
    check_lora(*lora_case(M + L, M, N, K, L, r, mixed))


@pytest.mark.parametrize("M,N,K,L,r", [
    (130, 4224, 384, 3, 40), (300, 8320, 256, 60, 16), (1100, 8448, 256, 30, 24),
    (1500, 384, 640, 50, 128), (2100, 640, 1152, 7, 48), (4093, 128, 128, 64, 8)])
def test_lora_add_planned(M, N, K, L, r):
    check_lora(*lora_case(M + L, M, N, K, L, r, True))


@pytest.mark.parametrize("M", [60, 400, 2100])
def test_lora_one_adapter_takes_most_rows_and_rows_that_are_not_finite_stay_alone(M):
    y, x, ad, ids = lora_case(5, M, 640, 512, 60, 32, False)
    ids[: M * 9 // 10] = 7
    want = check_lora(y, x, ad, ids)
    x[3, 9] = math.nan
    x[M - 1, 100] = math.inf
    got = eg.lora_add(y, x, ad, ids)
    other = torch.ones(M, dtype=torch.bool, device=DEV)
    other[[3, M - 1]] = False
    assert torch.equal(got[other], want[other])
    assert torch.isnan(got[3].float()).all()


@pytest.mark.parametrize("M", [400, 2100])
def test_lora_unused_ranks_of_a_planned_batch(M):
    y, x, ad, ids = lora_case(6, M, 256, 256, 50, 40, False)
    n = 37
    A, B = ad.A.clone(), ad.B.clone()
    A[:, n:] = math.nan
    B[:, :, n:] = math.inf
    ranks = torch.full((50,), n, dtype=torch.int32, device=DEV)
    ranks[::7] = 0
    got = check_lora(y, x, eg.LoraAdapters(A, B, ad.scale, ranks), ids)
    assert torch.isfinite(got.float()).all()


def test_lora_workspace_of_a_larger_batch():
    y, x, ad, ids = lora_case(8, 2100, 256, 384, 50, 16, True)
    ws = eg.lora_workspace(2100, 256, 384, ad, DEV)
    for M in (2100, 1200, 600, 130, 128, 1):
        check_lora(y[:M], x[:M], ad, ids[:M], workspace=ws)


def test_lora_in_place_odd_ids_and_unused_ranks():
    y, x, ad, ids = lora_case(3, 50, 256, 256, 4, 16, False)
    ids[::5] = -7
    ids[1::5] = 4
    ids[2::5] = 2 ** 31 - 1
    want = check_lora(y, x, ad, ids)
    got = y.clone()
    assert eg.lora_add(got, x, ad, ids, out=got) is got
    assert torch.equal(got, want)
    # what lies past an adapter's rank is not read as numbers
    A, B = ad.A.clone(), ad.B.clone()
    A[:, 5:] = math.nan
    B[:, :, 5:] = math.inf
    for n in (1, 2, 3, 4, 5):
        odd = eg.LoraAdapters(A, B, ad.scale,
                              torch.tensor([n, 5, 0, -3], dtype=torch.int32, device=DEV))
        got = check_lora(y, x, odd, ids)
        assert torch.isfinite(got.float()).all()
        keep = (ids == 2) | (ids == 3)
        assert torch.equal(got[keep], y[keep])
    # ranks beyond r count as r
    over = eg.LoraAdapters(ad.A, ad.B, ad.scale,
                           torch.full((4,), 99, dtype=torch.int32, device=DEV))
    assert torch.equal(eg.lora_add(y, x, over, ids), want)
    none = torch.full_like(ids, -1)
    assert torch.equal(eg.lora_add(y, x, ad, none), y)
    assert eg.lora_add(y[:0], x[:0], ad, ids[:0]).shape == (0, 256)


def test_lora_repeats_and_streams():
    y, x, ad, ids = lora_case(4, 100, 512, 512, 6, 32, True)
    ws = eg.lora_workspace(100, 512, 512, ad, DEV)
    ws.fill_(0xFF)
    want = check_lora(y, x, ad, ids, workspace=ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    outs = [eg.lora_add(y, x, ad, ids, workspace=ws, stream=st) for _ in range(3)]
    st.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("M", [1, 5, 33, 200])
def test_w4a8_linear_lora(M):
    N, K, L, r = 384, 512, 5, 16
    _, x, ad, ids = lora_case(M, M, N, K, L, r, True)
    packed = eg.pack_w4(*w4(gen(M), N, K))
    base = eg.w4a8_linear(x, packed, N)
    got = eg.w4a8_linear_lora(x, packed, N, ad, ids)
    ref, bound = lora_ref(base, x, ad, ids)
    assert ((got.double() - ref).abs() <= bound).all()


# ------------------------------------------------ inputs that change between calls ---
# Kernels that begin before the one in front of them has ended must still see
# what was written just before the call, and not what the last call left.

@pytest.mark.parametrize("M", [1, 5, 100, 260, 1300])
def test_w4a8_linear_lora_follows_inputs_rewritten_in_place(M):
    N, K, L, r = 512, 768, 20, 24
    cases = [lora_case(20 + i, M, N, K, L, r, True) for i in range(3)]
    packed = eg.pack_w4(*w4(gen(1), N, K))
    ad = cases[0][2]
    x, ids = torch.empty_like(cases[0][1]), torch.empty_like(cases[0][3])
    ws = eg.w4a8_linear_lora_workspace(M, N, K, ad, DEV)
    want = []
    for _, xi, _, idi in cases:
        y = eg.w4a8_linear(xi, packed, N)
        want.append(eg.lora_add(y, xi, ad, idi))
        torch.cuda.synchronize()
    got = []
    for i in range(24):
        x.copy_(cases[i % 3][1])
        ids.copy_(cases[i % 3][3])
        got.append(eg.w4a8_linear_lora(x, packed, N, ad, ids, workspace=ws))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 3]), i
    assert eg.device_status() == 0


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("T,path", [(1, eg.PATH_AUTO), (7, eg.PATH_AUTO), (30, eg.PATH_GEMV),
                                    (90, eg.PATH_TC), (900, eg.PATH_TC)])
def test_experts_follow_inputs_rewritten_in_place(variant, T, path):
    E, k, H, I = 8, 2, 512, 256
    cases = [experts_case(30 + i, T, E, k, H, I) for i in range(3)]
    layer = eg.moe_pack(*cases[0][3], *cases[0][4])
    x, ids, w = (torch.empty_like(t) for t in cases[0][:3])
    ws = eg.moe_workspace(T, k, E, H, I, variant, DEV, path)
    want = []
    for c in cases:
        want.append(eg.moe_experts(*c[:3], layer, variant=variant, path=path))
        torch.cuda.synchronize()
    got = []
    for i in range(24):
        for to, new in zip((x, ids, w), cases[i % 3][:3]):
            to.copy_(new)
        got.append(eg.moe_experts(x, ids, w, layer, variant=variant, path=path, workspace=ws))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 3]), i
    assert eg.device_status() == 0


# ------------------------------------------------------- offsets past 32 bits ---

def some_rows(n):
    return torch.cat([torch.arange(8), torch.randint(0, n, (200,)),
                      torch.arange(n - 200, n)]).to(DEV)


def test_lora_of_more_than_2_to_the_31_outputs():
    M, N = 120000, 18944
    y, x, ad, ids = lora_case(1, M, N, 256, 8, 16, True)
    got = eg.lora_add(y, x, ad, ids)
    rows = some_rows(M)
    ref, bound = lora_ref(y[rows], x[rows], ad, ids[rows])
    assert ((got[rows].double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("variant", VARIANTS)
def test_experts_of_more_than_2_to_the_31_sorted_values(variant):
    T, E, k, H, I = 300000, 4, 4, 2048, 128
    x, ids, w, gu, dn = experts_case(2, T, E, k, H, I)
    y = eg.moe_experts(x, ids, w, eg.moe_pack(*gu, *dn), variant=variant)
    rows = some_rows(T)
    ref, bound = experts_ref(x[rows], ids[rows], w[rows], gu, dn, variant)
    assert ((y[rows].double() - ref).abs() <= bound).all()
    assert eg.device_status() == 0
