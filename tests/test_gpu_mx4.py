"""Microscaled 4-bit linears on the GPU against their definition in 64 bits
(tests/mx4_helpers.py)."""
import math

import pytest
import torch

import w4a8_quantized_gemm_gb300 as eg
from mx4_helpers import BLOCK, dequant, quant, same_codes, tolerance, values_in

pytestmark = pytest.mark.gpu

FORMATS = [eg.MX4_E8M0, eg.MX4_E4M3]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def tscale(x, fmt):
    return (x.float().abs().max() / 2688.0).reshape(1) if fmt == eg.MX4_E4M3 else None


def weight(g, fmt, *shape):
    """A packed weight and its 64-bit values [.., N, K] (scaled)."""
    w = rand(g, *shape, scale=0.05, dtype=torch.float32)
    sets = shape[0] if len(shape) == 3 else 1
    ts = None
    if fmt == eg.MX4_E4M3:
        ts = w.reshape(sets, -1).abs().amax(dim=1) / 2688.0
    u = w if ts is None else w / (ts.view(sets, 1, 1) if len(shape) == 3 else ts)
    c, s = quant(u.reshape(-1, shape[-1]).double(), fmt)
    c, s = c.view(*shape[:-1], -1), s.view(*shape[:-1], -1)
    v = dequant(c, s, fmt)
    if ts is not None:
        v = v * (ts.double().view(sets, 1, 1) if len(shape) == 3 else ts.double())
    return eg.mx4_pack(c, s, fmt, tensor_scale=ts), v, (c, s)


def rows64(x, K, fmt, ts, gated=False):
    v = dequant(*quant(values_in(x, K, fmt, ts, gated), fmt), fmt)
    return v if ts is None else v * ts.double()


def check(y, a, w):
    """y against a [M, K] times w [N, K]."""
    ref = a @ w.t()
    off = (y.double() - ref).abs()
    bad = off > tolerance(ref, a.abs() @ w.abs().t(), a.shape[1], y.dtype)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, {off.max()}"


# --------------------------------------------------------------- quantization ---

def awkward(g, M, K, dtype):
    """Blocks of every size a type has, zeros, ties, a lone large value."""
    x = torch.randn(M, K, generator=g, device="cuda")
    e = torch.randint(-24 if dtype is torch.float16 else -140, 10, (M, K // 16), generator=g,
                      device="cuda")
    x = x * torch.ldexp(torch.ones((), device="cuda", dtype=torch.float64),
                        e).repeat_interleave(16, dim=1)
    x[::3, : K // 2] = (torch.randint(-24, 25, (len(x[::3]), K // 2), generator=g, device="cuda")
                        * 0.25).double()
    x[1::5, 16:32] = 0.0
    x[2::7, 0] = 30000.0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (130, 288), (259, 1056), (1, 18944),
                                 (1811, 2336)])
def test_codes_and_scales(fmt, dtype, M, K):
    x = awkward(gen(1), M, K, dtype)
    rows = eg.mx4_quant(x, fmt)
    c, s = quant(x.double(), fmt)
    assert torch.equal(rows.scales, s)
    assert same_codes(rows.codes, c)
    # the products' form holds the same
    c2, s2 = eg.mx4_unpack(eg.Mx4Weight(rows.a_tc, 0, M, K, fmt, None))
    assert torch.equal(s2, rows.scales) and torch.equal(c2, rows.codes)
    assert eg.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [1.0, 0.0117, 3.0e-5, 1000.0, -0.02])
def test_tensor_scale(dtype, scale):
    x = awkward(gen(2), 67, 480, dtype)
    ts = torch.tensor([scale], device="cuda")
    rows = eg.mx4_quant(x, eg.MX4_E4M3, tensor_scale=ts)
    c, s = quant(values_in(x, 480, 1, ts, False), eg.MX4_E4M3)
    assert torch.equal(rows.scales, s) and same_codes(rows.codes, c)
    v = dequant(rows.codes, rows.scales, eg.MX4_E4M3) * ts.double()
    for out in TYPES:
        got = eg.mx4_dequant(rows, dtype=out)
        assert torch.equal(got, v.float().to(out))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_values_back(fmt, dtype):
    """Every code under every scale, exactly."""
    top = 255 if fmt == eg.MX4_E8M0 else 128
    n = BLOCK[fmt]
    scales = torch.arange(top, dtype=torch.uint8, device="cuda").repeat_interleave(32 // n)
    K = top * 32
    codes = (torch.arange(K // 2, device="cuda") * 37 % 256).to(torch.uint8).view(1, -1)
    rows = eg.Mx4Rows(codes, scales.view(1, -1), None, 1, K, fmt, None)
    want = dequant(codes, scales.view(1, -1), fmt).float().to(dtype)
    assert torch.equal(torch.nan_to_num(eg.mx4_dequant(rows, dtype=dtype), nan=7.5),
                       torch.nan_to_num(want, nan=7.5))


@pytest.mark.parametrize("fmt", FORMATS)
def test_blocks_without_a_value(fmt):
    x = rand(gen(3), 4, 128, dtype=torch.float32)
    n = BLOCK[fmt]
    x[0, 5], x[1, n + 1], x[2, 2 * n] = math.nan, math.inf, -math.inf
    rows = eg.mx4_quant(x, fmt)
    v = eg.mx4_dequant(rows, dtype=torch.float32)
    nan = torch.zeros(4, 128, dtype=torch.bool, device="cuda")
    nan[0, :n] = nan[1, n:2 * n] = nan[2, 2 * n:3 * n] = True
    assert torch.equal(v.isnan(), nan)
    assert torch.equal(rows.scales[3], quant(x[3:].double(), fmt)[1][0])
    # a row that holds one gives NaN, its neighbours do not
    w, w64, _ = weight(gen(4), fmt, 40, 128)
    y = eg.mx4_linear(x, w)
    assert y[:3].isnan().all()
    check(y[3:], rows64(x[3:], 128, fmt, None), w64)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (33, 1056), (2600, 1408)])
def test_gated_codes(fmt, dtype, M, K):
    """Codes of the real gated values: none of 64 bits' is off by rounding."""
    g = gen(5)
    x = rand(g, M, 2 * K, scale=2.5, dtype=dtype)
    x[::4, :16] = 0.0
    # large gates: the gated value is next to a product of short numbers
    x[1::4, 32:64] = (torch.randint(8, 40, (len(x[1::4]), min(32, 2 * K - 32)), generator=g,
                                    device="cuda").to(dtype))
    ts = torch.tensor([0.013], device="cuda") if fmt == eg.MX4_E4M3 else None
    rows = eg.mx4_quant(x, fmt, tensor_scale=ts, gated=True)
    c, s = quant(values_in(x, K, fmt, ts, True), fmt)
    assert torch.equal(rows.scales, s) and same_codes(rows.codes, c)


@pytest.mark.parametrize("fmt", FORMATS)
def test_gated_values_where_fp32_runs_out(fmt):
    """Gates far below zero, tiny products, a tensor scale that makes up for them."""
    K = 64
    x = torch.zeros(6, 2 * K, device="cuda")
    i = torch.arange(K, device="cuda")
    x[0, :K], x[0, K:] = -85.0 - 0.25 * i, 1e30
    x[1, :K], x[1, K:] = 1e-25, 1e-20 * (1 + i)
    x[2, :K], x[2, K:] = -60.0 - i, 1.0
    x[3, :K], x[3, K:] = 1e-30 * (1 + i), 1e-15
    x[4, :K], x[4, K:] = 3.0e30, 1e6
    x[4, 40], x[4, K + 40] = 3e30, 3e30          # beyond fp32
    x[5, ::3] = 1.0
    ts = torch.tensor([1e-30], device="cuda") if fmt == eg.MX4_E4M3 else None
    if ts is not None:
        x[4] = 0.0
    rows = eg.mx4_quant(x, fmt, tensor_scale=ts, gated=True)
    c, s = quant(values_in(x, K, fmt, ts, True), fmt)
    assert torch.equal(rows.scales, s) and same_codes(rows.codes, c)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("low,high", [(-40.0, -22.0), (-24.0, -8.0), (-8.0, 30.0)])
def test_gated_values_next_to_borders(fmt, low, high):
    """Values within 2^-17 of a border between two codes, or (alone in their block)
    between two scales: fp32 may not decide what it cannot tell."""
    g, M, K = gen(24), 2048, 512
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda",
                          dtype=torch.float64)
    gate = (torch.rand(M, K, generator=g, device="cuda") * (high - low) + low)
    near = 1.0 + (torch.rand(M, K, generator=g, device="cuda").double() * 2 - 1) * 2.0 ** -17
    want = border[torch.randint(0, 7, (M, K), generator=g, device="cuda")] * near
    # the first of a block: 6 (a scale of 1), or the block's only value
    first, alone = slice(0, K, BLOCK[fmt]), torch.arange(M, device="cuda") % 2 == 0
    want[:, first] = 6.0
    gate[:, first] = 24.0
    lone = torch.zeros_like(want)
    # 4, or 6 * 1.0625, which lies between two e4m3 numbers
    lone[:, first] = (4.0 if fmt == eg.MX4_E8M0 else 6.375) * near[:, first]
    want = torch.where(alone[:, None], lone, want)
    lone_gate = torch.rand(M, K, generator=g, device="cuda") * (high - low) + low
    gate = torch.where(alone[:, None], lone_gate, gate)
    silu = gate.double() / (1.0 + torch.exp(-gate.double()))
    up = (want / silu).float()
    x = torch.cat([gate, up], dim=1)
    r = eg.mx4_quant(x, fmt, gated=True)
    codes, scales = quant(values_in(x, K, fmt, None, True), fmt)
    assert torch.equal(r.scales, scales)
    assert same_codes(r.codes, codes)


# -------------------------------------------------------------------- products ---

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 128, 256), (2, 130, 64), (7, 200, 96), (16, 256, 512), (17, 127, 288),
    (64, 384, 1056), (65, 33, 320), (128, 129, 2048), (129, 257, 768), (300, 500, 1312),
    (1, 3584, 3584), (5, 512, 18944), (517, 1031, 2080)])
def test_linear(fmt, M, N, K):
    g = gen(M * 7 + N)
    x = rand(g, M, K)
    w, w64, _ = weight(g, fmt, N, K)
    ts = tscale(x, fmt)
    y = eg.mx4_linear(x, w, tensor_scale=ts)
    assert eg.device_status() == 0
    check(y, rows64(x, K, fmt, ts), w64)
    # in two calls, the same
    rows = eg.mx4_quant(x, fmt, tensor_scale=ts, with_codes=False)
    assert torch.equal(eg.mx4_gemm(rows, w), y)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(250, 4112, 1376), (1150, 2192, 1056), (1000, 20480, 96),
                                   (510, 20640, 288), (1150, 2200, 1056), (1021, 3584, 544),
                                   (131, 20000, 160), (545, 19200, 800), (2048, 3600, 352)])
def test_many_rows(fmt, dtype, M, N, K):
    """Last tiles of every kind, odd blocks of weights and of rows, y off a boundary of
    32 bytes."""
    g = gen(M + N)
    x = rand(g, M, K, dtype=dtype)
    w, w64, _ = weight(g, fmt, N, K)
    ts = tscale(x, fmt)
    a64 = rows64(x, K, fmt, ts)
    room = torch.full((M * N + 32,), 7.0, dtype=dtype, device="cuda")
    for at in (0, 16 // room.element_size()):
        y = room[at: at + M * N].view(M, N)
        eg.mx4_linear(x, w, tensor_scale=ts, out=y)
        check(y, a64, w64)
        assert (room[at + M * N:] == 7.0).all()
        rows = eg.mx4_quant(x, fmt, tensor_scale=ts, with_codes=False)
        assert torch.equal(eg.mx4_gemm(rows, w, dtype=dtype), y)
    assert eg.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("x_type", TYPES)
@pytest.mark.parametrize("y_type", TYPES)
def test_types(fmt, x_type, y_type):
    g = gen(11)
    x = rand(g, 37, 416, dtype=x_type)
    w, w64, _ = weight(g, fmt, 201, 416)
    y = eg.mx4_linear(x, w, dtype=y_type)
    assert y.dtype is y_type
    check(y, rows64(x, 416, fmt, None), w64)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 384, 1408), (3, 1000, 4512), (16, 130, 288), (40, 200, 96),
                                   (259, 130, 512)])
def test_gated_linear(fmt, dtype, M, N, K):
    """Quantized by the product's kernel (few rows) or apart: the same codes."""
    g = gen(12)
    x = rand(g, M, 2 * K, scale=1.5, dtype=dtype)
    x[:, :8] = -50.0
    ts = torch.tensor([0.004], device="cuda") if fmt == eg.MX4_E4M3 else None
    w, w64, _ = weight(g, fmt, N, K)
    y = eg.mx4_linear(x, w, tensor_scale=ts, gated=True)
    check(y, rows64(x, K, fmt, ts, gated=True), w64)
    rows = eg.mx4_quant(x, fmt, tensor_scale=ts, gated=True, with_codes=False)
    assert torch.equal(eg.mx4_gemm(rows, w, dtype=dtype), y)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(1, 40000, 288), (9, 640, 1824), (16, 33, 2048), (17, 33, 2048)])
def test_few_rows_are_the_same_either_way(fmt, dtype, M, N, K):
    """mx4_linear of few rows quantizes them in the product's kernel."""
    g = gen(14)
    x = awkward(g, M, K, dtype)
    x[0, 3] = math.inf
    w, _, _ = weight(g, fmt, N, K)
    ts = torch.tensor([0.37], device="cuda") if fmt == eg.MX4_E4M3 else None
    rows = eg.mx4_quant(x, fmt, tensor_scale=ts)
    y, z = eg.mx4_linear(x, w, tensor_scale=ts, dtype=torch.float32), eg.mx4_gemm(
        rows, w, dtype=torch.float32)
    assert torch.equal(torch.nan_to_num(y, nan=1e30), torch.nan_to_num(z, nan=1e30))
    assert y[0].isnan().all() and not y[1:].isnan().any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_pack_and_back(fmt):
    for shape in [(1, 32), (130, 288), (3, 129, 96)]:
        w, _, (c, s) = weight(gen(13), fmt, *shape)
        c2, s2 = eg.mx4_unpack(w)
        assert torch.equal(c, c2) and torch.equal(s, s2)


# --------------------------------------------------------------- ragged products ---

def check_ragged(counts, N, K, fmt, before=0, after=0, tokens=None, gated=False, seed=20,
                 dtype=torch.bfloat16):
    g = gen(seed)
    E, n = len(counts), before + sum(counts) + after
    off = before + torch.tensor([0] + counts, device="cuda").cumsum(0)
    x = rand(g, tokens or n, K * (2 if gated else 1), dtype=dtype)
    index = None
    if tokens:
        index = torch.randint(0, tokens, (n,), generator=g, device="cuda", dtype=torch.int32)
    w, w64, _ = weight(g, fmt, E, N, K)
    ts = tscale(x, fmt)
    y = torch.full((n, N), 77.0, dtype=dtype, device="cuda")
    eg.mx4_linear_ragged(x, off.int(), w, index=index, tensor_scale=ts, gated=gated, out=y)
    assert eg.device_status() == 0
    a = rows64(x, K, fmt, ts, gated)
    if tokens:
        a = a[index.long()]
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo < hi:
            check(y[lo:hi], a[lo:hi], w64[e])
    assert (y[:before] == 77.0).all() and (y[n - after:] == 77.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,N,K", [
    ([1], 32, 32), ([0, 0, 3], 130, 96), ([5, 0, 1, 16, 17], 256, 512),
    ([127, 128, 129, 1, 0, 300], 200, 288), ([0] * 40 + [2] + [0] * 40, 64, 256),
    ([3] * 33, 100, 64), ([700, 20], 384, 1056)])
def test_ragged(fmt, counts, N, K):
    check_ragged(counts, N, K, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sets,rows", [(1024, 700), (1024, 70000), (33, 31), (65, 65 * 64 + 1)])
def test_many_sets(fmt, sets, rows):
    g = torch.Generator().manual_seed(sets + rows)
    counts = torch.bincount(torch.randint(0, sets, (rows,), generator=g), minlength=sets)
    check_ragged(counts.tolist(), 24, 64, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_ragged_gathered_and_gated(fmt):
    check_ragged([9, 0, 150, 30], 257, 480, fmt, tokens=50)
    check_ragged([9, 0, 150, 30], 257, 480, fmt, tokens=300)
    # many from few: quantized once, gathered in 4 bits
    check_ragged([9, 0, 11900, 300, 33], 130, 1056, fmt, tokens=1900, before=2, after=1)
    check_ragged([4, 2900, 0, 30], 33, 4512, fmt, tokens=11, gated=True, before=2, after=1)
    check_ragged([9, 0, 150, 30], 257, 480, fmt, gated=True)
    check_ragged([2, 0, 3], 64, 96, fmt, before=4, after=130)
    check_ragged([2, 0, 3], 64, 96, fmt, before=1, after=2, tokens=3, gated=True,
                 dtype=torch.float16)
    for counts in ([0, 1, 0, 1, 1, 0], [16], [1] * 8):
        check_ragged(counts, 300, 1056, fmt, tokens=2)
        check_ragged(counts, 300, 1056, fmt, gated=True, before=1, dtype=torch.float32)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,n,K", [(6, 20, 96), (20, 20, 96), (30, 12300, 1056)])
def test_index_outside_reads_zeros(fmt, tokens, n, K):
    g = gen(23)
    x = rand(g, tokens, K)
    index = torch.arange(n, device="cuda", dtype=torch.int32) % tokens
    index[3], index[11], index[n - 1] = -1, tokens, 2 ** 31 - 1
    w, w64, _ = weight(g, fmt, 2, 40, K)
    off = torch.tensor([0, 7, n], dtype=torch.int32, device="cuda")
    y = eg.mx4_linear_ragged(x, off, w, index=index)
    ok = (index >= 0) & (index < tokens)
    assert (y[~ok] == 0).all()
    a = rows64(x, K, fmt, None)[torch.where(ok, index, 0).long()] * ok[:, None]
    for e, (lo, hi) in enumerate(((0, 7), (7, n))):
        check(y[lo:hi], a[lo:hi], w64[e])


@pytest.mark.parametrize("bad", [
    [0, 5, 3, 10, 10], [-4, 2, 2, 9, 12], [0, 99, 99, 99, 99], [20, 1, 2, 3, 4], [5, 5, 5, 5, 5]])
def test_offsets_out_of_order_or_range_count_as_the_nearest(bad):
    """What the header says of them: rising, within [0, rows]."""
    g = gen(24)
    x = rand(g, 12, 64)
    w, w64, _ = weight(g, 0, 4, 40, 64)
    y = torch.full((12, 40), 9.0, dtype=torch.bfloat16, device="cuda")
    eg.mx4_linear_ragged(x, torch.tensor(bad, dtype=torch.int32, device="cuda"), w, out=y)
    off = torch.tensor(bad).clamp(0, 12).cummax(0).values.tolist()
    a = rows64(x, 64, 0, None)
    for e in range(4):
        if off[e] < off[e + 1]:
            check(y[off[e]:off[e + 1]], a[off[e]:off[e + 1]], w64[e])
    assert (y[:off[0]] == 9.0).all() and (y[off[4]:] == 9.0).all()


# ------------------------------------------------------ streams, graphs, sharing ---

def test_another_stream_and_no_workspace():
    g = gen(30)
    w, w64, _ = weight(g, 1, 300, 512)
    s = torch.cuda.Stream()
    for M in (1, 40, 200):
        x = rand(g, M, 512)
        ts = tscale(x, 1)
        s.wait_stream(torch.cuda.current_stream())
        y = eg.mx4_linear(x, w, tensor_scale=ts, stream=s)
        rows = eg.mx4_quant(x, 1, tensor_scale=ts, stream=s)
        z = eg.mx4_gemm(rows, w, stream=s)
        v = eg.mx4_dequant(rows, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        check(y, rows64(x, 512, 1, ts), w64)
        assert torch.equal(y, z)
        assert torch.equal(v.double(), rows64(x, 512, 1, ts).float().bfloat16().double())


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_and_replayed_with_other_rows(fmt):
    """One graph of a dense and a ragged call; offsets, index and rows change between
    replays, within the sizes."""
    g = gen(31)
    n, K, N, E, T = 600, 576, 200, 6, 90
    w, w64, _ = weight(g, fmt, E, N, K)
    d, d64, _ = weight(g, fmt, N, K)
    x, ts = rand(g, T, K), (torch.tensor([0.002], device="cuda") if fmt else None)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    index = torch.zeros(n, dtype=torch.int32, device="cuda")
    y = torch.zeros(n, N, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    ws, wd = eg.mx4_workspace(n, w, "cuda"), eg.mx4_workspace(T, d, "cuda")

    def call():
        eg.mx4_linear(x, d, tensor_scale=ts, out=z, workspace=wd)
        eg.mx4_linear_ragged(x, off, w, index=index, tensor_scale=ts, out=y, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for counts in ([100] * 6, [0, 0, 600, 0, 0, 0], [3, 0, 1, 250, 0, 90], [0] * 6):
        x.copy_(rand(g, T, K))
        off.copy_(torch.tensor([0] + counts).cumsum(0))
        index.copy_(torch.randint(0, T, (n,), generator=g, device="cuda"))
        y.fill_(3.0)
        graph.replay()
        a = rows64(x, K, fmt, ts)
        check(z, a, d64)
        lo = 0
        for e, c in enumerate(counts):
            if c:
                check(y[lo:lo + c], a[index[lo:lo + c].long()], w64[e])
            lo += c
        assert (y[lo:] == 3.0).all()
    assert eg.device_status() == 0


def test_two_calls_at_once_and_results_that_do_not_depend_on_timing():
    g = gen(32)
    w, _, _ = weight(g, 0, 1500, 4096)
    xs = [rand(g, m, 4096) for m in (1, 3, 70, 400)]
    want = [eg.mx4_linear(x, w) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for x, s in zip(xs, streams):
            got.append(eg.mx4_linear(x, w, stream=s))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % len(xs)])
    assert eg.device_status() == 0


def test_smaller_batches_share_a_workspace():
    g = gen(33)
    w, w64, _ = weight(g, 0, 3, 130, 320)
    ws = eg.mx4_workspace(500, w, "cuda")
    for counts in ([200, 100, 200], [0, 3, 0], [64, 65, 1], [1, 1, 1]):
        n = sum(counts)
        x = rand(g, n, 320)
        off = torch.tensor([0] + counts, device="cuda").cumsum(0)
        y = eg.mx4_linear_ragged(x, off.int(), w, workspace=ws)
        a = rows64(x, 320, 0, None)
        for e in range(3):
            if counts[e]:
                check(y[off[e]:off[e + 1]], a[off[e]:off[e + 1]], w64[e])


@pytest.mark.parametrize("fmt", FORMATS)
def test_output_past_2_31_values(fmt):
    """65,600 rows of 33,000 columns: places past 2^31, checked in the last rows."""
    g = gen(34)
    M, N, K = 65600, 33000, 64
    x = rand(g, M, K)
    w, w64, _ = weight(g, fmt, N, K)
    y = eg.mx4_linear(x, w)
    for rows in (slice(0, 3), slice(M - 40, M)):
        check(y[rows], rows64(x[rows], K, fmt, None), w64)


def test_experts_of_a_layer():
    """The run of a layer: route, rows sorted by expert, gate and up, gated down, sum."""
    g = gen(35)
    T, E, k, H, I = 75, 8, 3, 288, 160
    x = rand(g, T, H)
    gate_up, gu64, _ = weight(g, 0, E, 2 * I, H)
    down, d64, _ = weight(g, 0, E, H, I)
    weights, ids = eg.moe_route(rand(g, T, E, dtype=torch.float32), k)
    key, order = torch.sort(ids.view(-1), stable=True)
    off = torch.searchsorted(key, torch.arange(E + 1, device="cuda", dtype=torch.int32)).int()
    token = (order // k).int()
    h = eg.mx4_linear_ragged(x, off, gate_up, index=token)
    out = eg.mx4_linear_ragged(h, off, down, gated=True)
    y = torch.zeros(T, H, device="cuda").index_add_(
        0, token.long(), out.float() * weights.view(-1)[order][:, None])
    # each product against 64 bits from what it was given
    a, b = rows64(x, H, 0, None)[token.long()], rows64(h, I, 0, None, gated=True)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo < hi:
            check(h[lo:hi], a[lo:hi], gu64[e])
            check(out[lo:hi], b[lo:hi], d64[e])
    want.index_add_(0, token.long(), out.double() * weights.view(-1)[order].double()[:, None])
    assert ((y.double() - want).abs() <= 8 * 2.0 ** -24 * out.double().abs().max()).all()


def test_debug_build_checks_weight_records(monkeypatch):
    """Clean, and with the packed weight declared shorter than its buffer (the
    redirected reads stay inside it)."""
    monkeypatch.setattr(eg, "LIB_PATH", eg.DEBUG_LIB_PATH)
    monkeypatch.setattr(eg, "_lib", None)
    lib = eg.load()
    try:
        assert lib.egopq_debug_build() == 1
        g = gen(36)
        w, w64, _ = weight(g, 0, 300, 544)
        for M in (2, 40, 200):
            x = rand(g, M, 544)
            check(eg.mx4_linear(x, w), rows64(x, 544, 0, None), w64)
            assert eg.device_status() == 0
        lib.egopq_debug_set_record_limit(2 * 17408)
        eg.mx4_linear(rand(g, 2, 544), w)
        assert eg.device_status() == -7
    finally:
        lib.egopq_debug_set_record_limit(0)
        eg.device_status()


def test_ragged_without_rows():
    w, _, _ = weight(gen(21), 0, 4, 64, 64)
    x = rand(gen(22), 6, 64)
    y = torch.full((6, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    eg.mx4_linear_ragged(x, torch.zeros(5, dtype=torch.int32, device="cuda"), w, out=y)
    assert (y == 5.0).all()
    assert eg.mx4_linear_ragged(x[:0], torch.zeros(5, dtype=torch.int32, device="cuda"),
                                w).shape == (0, 64)
    assert eg.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_tensors_elsewhere_and_weights_too_short_are_refused(fmt):
    # (a weight put together by hand, or moved to the host with its fields)
    g = gen(23)
    w, _, _ = weight(g, fmt, 40, 64)
    many, _, _ = weight(g, fmt, 2, 40, 64)
    x, off = rand(g, 6, 64), torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    rows = eg.mx4_quant(x, fmt)
    bad = lambda t: [t._replace(packed=t.packed.cpu()), t._replace(packed=t.packed[:-16])]  # noqa: E731
    for v in bad(w):
        for call in (lambda: eg.mx4_linear(x, v), lambda: eg.mx4_gemm(rows, v),
                     lambda: eg.mx4_unpack(v)):
            with pytest.raises(ValueError, match="tensor (on|must be on)|needed"):
                call()
    for v in bad(many):
        with pytest.raises(ValueError, match="tensor on|needed"):
            eg.mx4_linear_ragged(x, off, v)
    y = torch.empty(6, 40, dtype=torch.bfloat16)
    ws = eg.mx4_workspace(6, many, "cuda").cpu()
    for call in (lambda: eg.mx4_linear(x, w, out=y), lambda: eg.mx4_linear(x, w, workspace=ws),
                 lambda: eg.mx4_linear_ragged(x, off.cpu(), many),
                 lambda: eg.mx4_linear_ragged(x, off, many, index=torch.zeros(6, dtype=torch.int32)),
                 lambda: eg.mx4_linear_ragged(x, off, many, workspace=ws),
                 lambda: eg.mx4_gemm(rows, w, out=y),
                 lambda: eg.mx4_gemm(rows._replace(a_tc=rows.a_tc.cpu()), w),
                 lambda: eg.mx4_dequant(rows._replace(scales=rows.scales.cpu())),
                 lambda: eg.mx4_quant(x, fmt, out=rows._replace(codes=rows.codes.cpu()))):
        with pytest.raises(ValueError, match="tensor (on|must be on)"):
            call()
    assert eg.device_status() == 0
