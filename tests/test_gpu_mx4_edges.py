"""Microscaled 4-bit linears at the ends of their types and between their kernels,
against the definition in 64 bits (tests/mx4_helpers.py)."""
import pytest
import torch

import w4a8_quantized_gemm_gb300 as eg
from mx4_helpers import BLOCK, quant, same_codes, values_in
from test_gpu_mx4 import FORMATS, gen

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------- quantization ---

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bits", [3, 10, 17, 23])
def test_gated_codes_of_subnormal_gates(fmt, bits):
    """fp32 gates of k steps of 2^-149, below 2^bits of them, with an up half that
    brings their product (times the tensor's scale, which e4m3 blocks need for it) back
    to ordinary numbers: half a gate is no number of fp32's where k is odd, so the
    codes are those of the real product only if it is not formed there."""
    g, M, K = gen(40 + bits), 512, 512
    k = torch.randint(1, 2 ** bits, (M, K), generator=g, device="cuda", dtype=torch.int32)
    gate = k.view(torch.float32)  # (the pattern of k * 2^-149)
    assert torch.equal(gate.double(), k.double() * 2.0 ** -149)
    size = torch.randint(0, 6, (M, K // BLOCK[fmt]), generator=g, device="cuda")
    want = (0.3 + 5.7 * torch.rand(M, K, generator=g, device="cuda").double()) * (
        2.0 ** size.double()).repeat_interleave(BLOCK[fmt], dim=1) * 2.0 ** -60
    # in every second row the first of a block is its only value
    lone = torch.zeros(K, dtype=torch.bool, device="cuda")
    lone[::BLOCK[fmt]] = True
    want[::2, ~lone] = 0.0
    up = (want / (0.5 * gate.double())).float()
    assert torch.isfinite(up).all()
    sign = torch.randint(0, 2, (M, K), generator=g, device="cuda") * 2.0 - 1.0
    x = torch.cat([gate * sign, up], dim=1)
    ts = torch.tensor([2.0 ** -60], device="cuda") if fmt == eg.MX4_E4M3 else None
    rows = eg.mx4_quant(x, fmt, tensor_scale=ts, gated=True)
    codes, scales = quant(values_in(x, K, fmt, ts, True), fmt)
    assert torch.equal(rows.scales, scales)
    assert same_codes(rows.codes, codes)


# ---------------------------------------------------------- weights, right away ---

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 16, 40, 400])
def test_a_weight_quantized_right_in_front_of_its_product(fmt, M):
    """An operand as the weight of the next call, which begins to read weights before
    what is in front of it has ended: the same values as of mx4_pack."""
    g, N, K = gen(50 + M), 2560, 3584
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    for turn in range(4):
        w = (torch.randn(N, K, generator=g, device="cuda") * 0.05).bfloat16()
        rows = eg.mx4_quant(w, fmt)
        want = eg.mx4_linear(x, eg.mx4_pack(rows.codes, rows.scales, fmt))
        xr = eg.mx4_quant(x, fmt, with_codes=False)
        for call in (lambda: eg.mx4_linear(x, eg.Mx4Weight(rows.a_tc, 0, N, K, fmt, None)),
                     lambda: eg.mx4_gemm(xr, eg.Mx4Weight(rows.a_tc, 0, N, K, fmt, None))):
            call()
            torch.cuda.synchronize()
            rows.a_tc.fill_(255)  # (codes of -6 under NaN)
            torch.cuda.synchronize()
            eg.mx4_quant(w, fmt, out=rows)
            assert torch.equal(call(), want)
    assert eg.device_status() == 0


def test_a_weight_dequantized_right_in_front_of_its_product():
    g, M, N, K = gen(60), 64, 2560, 3584
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    rows = eg.mx4_quant((torch.randn(N, K, generator=g, device="cuda") * 0.05).bfloat16(),
                        with_tc=False)
    w = eg.mx4_dequant(rows)
    want = eg.bf16_gemm_twin(x, w)
    for turn in range(4):
        torch.cuda.synchronize()
        w.fill_(float("nan"))
        torch.cuda.synchronize()
        eg.mx4_dequant(rows, out=w)
        assert torch.equal(eg.bf16_gemm_twin(x, w), want)
    assert eg.device_status() == 0


# -------------------------------------------------------------------- products ---

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(16, 16384, 2048), (12, 19456, 2304), (9, 14336, 2048),
                                   (14, 9856, 1024), (12, 39040, 1280), (4, 58368, 3328)])
def test_one_call_and_two_add_up_alike(fmt, gated, M, N, K):
    """mx4_linear gives the values of mx4_quant and mx4_gemm, to the last bit of fp32:
    sizes where the kernel of many rows would add up the few rows in another order.
    (Blocks spread over 2^20, so that sums are rounded.)"""
    g = gen(M + N)

    def spread(*shape):
        v = torch.randn(shape, generator=g, device="cuda")
        e = torch.randint(-10, 11, (shape[0], shape[1] // 32), generator=g, device="cuda")
        return v * (2.0 ** e).repeat_interleave(32, dim=1)

    x = spread(M, 2 * K if gated else K).bfloat16()
    r = eg.mx4_quant((spread(N, K) * 0.05).bfloat16(), fmt, with_tc=False)
    packed = eg.mx4_pack(r.codes, r.scales, fmt)
    rows = eg.mx4_quant(x, fmt, gated=gated, with_codes=False)
    y = eg.mx4_linear(x, packed, gated=gated, dtype=torch.float32)
    assert torch.equal(eg.mx4_gemm(rows, packed, dtype=torch.float32), y)
    z = eg.mx4_linear(x.float(), packed, gated=gated)
    assert z.dtype is torch.float32 and torch.equal(z, y)


# --------------------------------------------------------------- ragged products ---

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,K", [(20, 96), (12300, 1056)])
def test_an_x_without_rows_reads_as_zeros(fmt, n, K):
    """Quantized directly, and (many rows of few) by a gather."""
    g = gen(70)
    r = eg.mx4_quant(torch.randn(2 * 40, K, generator=g, device="cuda"), fmt, with_tc=False)
    w = eg.mx4_pack(r.codes.view(2, 40, -1), r.scales.view(2, 40, -1), fmt)
    y = torch.full((n, 40), 3.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([1, 7, n - 2], dtype=torch.int32, device="cuda")
    index = torch.randint(-5, 5, (n,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    eg.mx4_linear_ragged(x, off, w, index=index, out=y)
    assert (y[1:n - 2] == 0).all() and (y[:1] == 3.0).all() and (y[n - 2:] == 3.0).all()
    assert eg.device_status() == 0


# ------------------------------------------------------------------------- types ---

def test_a_result_has_the_type_of_its_output():
    g = gen(71)
    x = torch.randn(6, 64, generator=g, device="cuda").bfloat16()
    rows = eg.mx4_quant(x)
    w = eg.mx4_pack(rows.codes, rows.scales)
    for call, shape in ((lambda **k: eg.mx4_dequant(rows, **k), (6, 64)),
                        (lambda **k: eg.mx4_gemm(rows, w, **k), (6, 6)),
                        (lambda **k: eg.mx4_linear(x, w, **k), (6, 6))):
        assert call().dtype is torch.bfloat16
        for t in (torch.float16, torch.float32):
            want, out = call(dtype=t), torch.empty(shape, dtype=t, device="cuda")
            assert want.dtype is t
            assert call(out=out) is out and torch.equal(out, want)
            assert call(dtype=t, out=out) is out and torch.equal(out, want)


# ------------------------------------------------------------------- debug build ---

@pytest.mark.parametrize("fmt", FORMATS)
def test_debug_build_checks_the_records_of_both_kernels(monkeypatch, fmt):
    """Of few rows and of many: a weight declared shorter than its buffer (to which the
    redirected reads keep) is noticed, and nothing is where it is whole."""
    monkeypatch.setattr(eg, "LIB_PATH", eg.DEBUG_LIB_PATH)
    monkeypatch.setattr(eg, "_lib", None)
    lib = eg.load()
    try:
        assert lib.egopq_debug_build() == 1
        g, record = gen(72), 17408 if fmt == eg.MX4_E8M0 else 18432
        r = eg.mx4_quant(torch.randn(300, 544, generator=g, device="cuda"), fmt, with_tc=False)
        w = eg.mx4_pack(r.codes, r.scales, fmt)
        assert w.packed.nbytes == 9 * record
        for M in (2, 40, 200, 700):
            x = torch.randn(M, 544, generator=g, device="cuda").bfloat16()
            lib.egopq_debug_set_record_limit(0)
            eg.mx4_linear(x, w)
            assert eg.device_status() == 0, M
            for records in (2, 8):
                lib.egopq_debug_set_record_limit(records * record)
                eg.mx4_linear(x, w)
                assert eg.device_status() == -7, (M, records)
    finally:
        lib.egopq_debug_set_record_limit(0)
        eg.device_status()
