"""Host checks of the microscaled 4-bit linears: refusals come before anything
touches a device (addresses here are never read), and the oracle's own checks."""
import pytest
import torch

import w4a8_quantized_gemm_gb300 as eg
from mx4_helpers import dequant, e4m3_table, magnitude, quant
from test_rows_cpu import lib  # noqa: F401

A = 1 << 20  # an aligned address that nothing reads
BIG = 1 << 40


def code(lib, rc, word):
    assert rc < 0 and word in lib.egopq_last_error_string().decode(), (
        rc, lib.egopq_last_error_string())
    return rc


def q(lib, x=A, x_type=0, M=4, K=64, fmt=0, ts=None, gated=0, c=A, s=A, op=A):
    return lib.egopq_mx4_quant(x, x_type, M, K, fmt, ts, gated, c, s, op, None)


def linear(lib, x=A, x_type=0, M=4, N=8, K=64, a=None, w=A, ws=None, fmt=0, y_type=0, y=2 * A,
           work=3 * A, nbytes=BIG):
    return lib.egopq_mx4_linear(x, x_type, M, N, K, 0, a, w, ws, fmt, y_type, y, work, nbytes, None)


def ragged(lib, x=A, x_rows=4, index=None, off=A, rows=4, sets=3, N=8, K=64, a=None, ws=None,
           fmt=0, y=2 * A, work=3 * A, nbytes=BIG):
    return lib.egopq_mx4_linear_ragged(x, 0, x_rows, index, off, rows, sets, N, K, 0, a, A, ws, fmt,
                                       0, y, work, nbytes, None)


def test_sizes(lib):
    # records of 128 rows and 256 K: 16384 bytes of codes, a byte a block of scales
    assert lib.egopq_mx4_operand_bytes(1, 32, 0) == 17408
    assert lib.egopq_mx4_operand_bytes(129, 288, 1) == 4 * 18432
    assert lib.egopq_mx4_packed_bytes(3, 130, 256, 0) == 6 * 17408
    assert lib.egopq_mx4_linear_workspace_bytes(128, 0, 256, 0) == 17408
    # each set with rows may begin a block of its own; and codes and scales of a
    # quarter as many rows, if the rows are gathered from so few
    assert lib.egopq_mx4_linear_workspace_bytes(300, 8, 256, 0) == 10 * 17408 + 75 * 136 + 16
    assert lib.egopq_mx4_linear_workspace_bytes(3, 8, 256, 0) == 3 * 17408 + 16
    for bad in ((0, 32, 0), (4, 48, 0), (4, 0, 0), (4, 32, 2), (-1, 32, 0), (1 << 31, 32, 0)):
        assert lib.egopq_mx4_operand_bytes(*bad) == 0, bad
    for bad in ((0, 8, 32, 0), (1025, 8, 32, 0), (1, 0, 32, 0), (1, 8, 31, 0), (1, 8, 32, -1)):
        assert lib.egopq_mx4_packed_bytes(*bad) == 0, bad
    assert lib.egopq_mx4_linear_workspace_bytes(4, 1025, 32, 0) == 0
    assert lib.egopq_mx4_linear_workspace_bytes(0, 2, 32, 0) == 0


def test_quantization_refuses(lib):
    assert q(lib, M=0, x=None) == 0
    assert code(lib, q(lib, K=48), "multiple of 32") == -2
    assert code(lib, q(lib, M=-1), "sizes") == -1
    assert code(lib, q(lib, M=1 << 31), "large") == -2
    assert code(lib, q(lib, fmt=2), "format") == -1
    assert code(lib, q(lib, x_type=3), "x_type") == -1
    assert code(lib, q(lib, x=None), "x is NULL") == -1
    assert code(lib, q(lib, x=A + 8), "x is not") == -3
    assert code(lib, q(lib, c=None), "together") == -1
    assert code(lib, q(lib, s=None), "together") == -1
    assert code(lib, q(lib, c=None, s=None, op=None), "neither") == -1
    assert code(lib, q(lib, op=A + 4), "operand") == -3
    assert code(lib, q(lib, ts=A), "no tensor scale") == -1
    assert code(lib, q(lib, fmt=1, ts=A + 2), "4-byte") == -3
    d = lib.egopq_mx4_dequant
    assert d(None, None, 0, 64, 0, None, 0, None, None) == 0
    assert code(lib, d(A, A, 4, 64, 0, None, 5, A, None), "y_type") == -1
    assert code(lib, d(A, None, 4, 64, 0, None, 0, A, None), "scales") == -1
    assert code(lib, d(A, A, 4, 64, 0, A, 0, A, None), "no tensor scale") == -1


def test_packing_refuses(lib):
    for f in (lib.egopq_mx4_pack, lambda c, s, *r: lib.egopq_mx4_unpack(r[4], *r[:4], c, s, None)):
        assert code(lib, f(A, A, 1, 8, 40, 0, A, None), "multiple of 32") == -2
        assert code(lib, f(A, A, 0, 8, 64, 0, A, None), "sizes") == -1
        assert code(lib, f(A, A, 1025, 8, 64, 0, A, None), "at most 1024") == -2
        assert code(lib, f(A, A, 1, 8, 64, 9, A, None), "format") == -1
        assert code(lib, f(None, A, 1, 8, 64, 0, A, None), "codes") == -1
        assert code(lib, f(A, A + 1, 1, 8, 64, 0, A, None), "scales") == -3


def test_products_refuse(lib):
    g = lib.egopq_mx4_gemm
    assert g(None, None, None, None, 0, 8, 64, 0, 0, None, None) == 0
    assert code(lib, g(A, A, None, None, 4, 8, 33, 0, 0, A, None), "multiple of 32") == -2
    assert code(lib, g(None, A, None, None, 4, 8, 64, 0, 0, A, None), "operand") == -1
    assert code(lib, g(A, A + 2, None, None, 4, 8, 64, 0, 0, A, None), "packed") == -3
    assert code(lib, g(A, A, None, A, 4, 8, 64, 0, 0, A, None), "no tensor scale") == -1
    assert code(lib, g(A, A, A, A, 4, 8, 64, 1, 7, A, None), "y_type") == -1
    assert linear(lib, M=0, x=None, y=None, work=None) == 0
    assert code(lib, linear(lib, N=0), "sizes") == -1
    assert code(lib, linear(lib, x_type=4), "x_type") == -1
    assert code(lib, linear(lib, work=None), "workspace") == -1
    assert code(lib, linear(lib, nbytes=17407), "17408 needed") == -1
    assert code(lib, linear(lib, work=A + 64), "overlaps") == -1
    assert code(lib, linear(lib, work=2 * A - 17408 + 16), "overlaps") == -1
    # y [4][8] of two bytes on x [4][64]
    for y in (A, A + 496, A - 48):
        assert code(lib, linear(lib, y=y), "y overlaps x") == -1
    assert code(lib, linear(lib, a=A), "no tensor scale") == -1
    assert code(lib, linear(lib, fmt=1, a=A + 1), "4-byte") == -3


def test_ragged_products_refuse(lib):
    assert ragged(lib, rows=0, x_rows=0, off=None) == 0
    assert code(lib, ragged(lib, off=None), "offsets") == -1
    assert code(lib, ragged(lib, off=A + 2), "offsets") == -3
    assert code(lib, ragged(lib, index=A + 1), "index") == -3
    assert code(lib, ragged(lib, x_rows=5), "no index") == -1
    assert code(lib, ragged(lib, x_rows=-1, index=A), "rows of x") == -1
    assert code(lib, ragged(lib, sets=0), "sizes") == -1
    assert code(lib, ragged(lib, sets=1025), "at most 1024") == -2
    assert code(lib, ragged(lib, nbytes=3 * 17408 + 15), "needed") == -1
    assert code(lib, ragged(lib, x=None), "x is NULL") == -1
    # slices of an index and of offsets, at any of their elements
    assert code(lib, ragged(lib, off=A + 4, index=A + 12, nbytes=0), "needed") == -1


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="format"):
        eg.mx4_quant(x, 3)
    with pytest.raises(TypeError):
        eg.mx4_quant(x.to(torch.int8))
    with pytest.raises(ValueError, match="odd"):
        eg.mx4_quant(x[:, :33].contiguous(), gated=True)
    with pytest.raises(eg.EgopqError, match="multiple of 32"):
        eg.mx4_quant(x[:, :48].contiguous())
    with pytest.raises(ValueError, match="CUDA"):
        eg.mx4_quant(x)
    w = eg.Mx4Weight(torch.zeros(17408, dtype=torch.uint8), 0, 8, 64, 0, None)
    many = w._replace(sets=2, packed=torch.zeros(34816, dtype=torch.uint8))
    with pytest.raises(ValueError, match="several sets"):
        eg.mx4_linear(x, many)
    with pytest.raises(ValueError, match="several sets"):
        eg.mx4_linear_ragged(x, torch.zeros(2, dtype=torch.int32), w)
    with pytest.raises(ValueError, match="shape"):
        eg.mx4_linear(x, w, gated=True)
    rows = eg.Mx4Rows(None, None, None, 4, 64, 0, None)
    with pytest.raises(ValueError, match="with_tc"):
        eg.mx4_gemm(rows, w)
    with pytest.raises(ValueError, match="K=96"):
        eg.mx4_gemm(rows._replace(K=96), w)
    with pytest.raises(ValueError, match="with_codes"):
        eg.mx4_dequant(rows)
    with pytest.raises(eg.EgopqError, match="no tensor scale"):
        eg.mx4_pack(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8),
                    tensor_scale=torch.ones(1))


# ------------------------------------------------------------------- the oracle ---

def test_oracle_rounds_to_the_nearest_number():
    """Codes against a search over all of them, away from ties; ties by hand."""
    v = torch.rand(2000, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 7
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    assert torch.equal(magnitude(v).long(), (v[:, None] - grid).abs().argmin(dim=1))
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 99.0], dtype=torch.float64)
    assert magnitude(ties).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7]
    t = e4m3_table()
    assert torch.equal(t, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double())


def test_oracle_by_hand():
    x = torch.zeros(2, 32, dtype=torch.float64)
    x[0, 0], x[0, 1], x[0, 2] = 6.0, -2.4, 0.26     # floor(log2 6) = 2: scale 1
    c, s = quant(x, 0)
    assert s.tolist() == [[127], [0]] and c[0, :2].tolist() == [0xC7, 0x01]
    assert dequant(c, s, 0)[0, :4].tolist() == [6.0, -2.0, 0.5, 0.0]
    c, s = quant(x, 1)                              # 6 / 6 = 1: e4m3 0x38
    assert s.tolist() == [[0x38, 0], [0, 0]]
    x[1, 3] = 2.0 ** -12                            # 2^-12 / 6 rounds to 0
    assert quant(x, 1)[1].tolist() == [[0x38, 0], [0, 0]]
    x[1, 3] = float("nan")
    assert quant(x, 0)[1].tolist() == [[127], [255]] and quant(x, 1)[1][1].tolist() == [127, 0]
