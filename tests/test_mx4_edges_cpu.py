"""Host checks of the microscaled 4-bit linears: which kernels let the next one begin
early (in the sources: no run shows a race for certain), and what is refused
(addresses here are never read)."""
import os
import re

import pytest
import torch

import w4a8_quantized_gemm_gb300 as eg
from test_mx4_cpu import A, code, linear, q, ragged
from test_rows_cpu import lib  # noqa: F401
from w4a8_quantized_gemm_gb300 import builder


def source(name):
    with open(os.path.join(builder.CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """What stands between the braces behind `head`."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError(head)


def test_what_makes_weights_lets_no_kernel_begin_before_its_end():
    """Products read weights in front of their wait."""
    text, api = source("mx4_quant.cu"), source("mx4_api.cu")
    assert "griddep_launch_dependents" not in body(text, "mx4_pack_kernel(uint8_t* codes")
    quant = body(text, "mx4_quant_kernel(const QuantParams p)")
    assert re.findall(r"if \(([^\n]*)\) griddep_launch_dependents", quant) == [
        "EARLY && threadIdx.x == 0"]
    assert quant.count("griddep_launch_dependents") == 1
    assert len(re.findall(r"return a\.early \? launch_quant_u<[^>]*, true>\(a, sms, st\)\s*"
                          r": launch_quant_u<[^>]*, false>\(a, sms, st\);", text)) == 2
    # an operand of the caller's is such a weight; a linear's own is read by its product
    assert "a.early = !operand;" in body(api, "int egopq_mx4_quant(")
    assert api.count("early = true") == 1 and "early = true" in body(api, "int run(")


def test_dense_weights_are_read_behind_the_wait():
    """Any kernel may write such a matrix (mx4_dequant lets the next one begin early)."""
    text = source("tc_kernel.cuh")
    at = text.index("load_weights(i);")
    before = text[text.rindex("} else {", 0, at):at]
    assert re.search(r"if constexpr \(C::kW16\) griddep_wait\(\);\s*const int n_pre", before)


# --------------------------------------------------------------------- arguments ---

def test_an_x_without_rows_needs_no_address(lib):  # noqa: F811
    # (every index is outside it; the workspace is the next thing to be looked at)
    assert code(lib, ragged(lib, x=None, x_rows=0, index=A, nbytes=0), "needed") == -1
    assert code(lib, ragged(lib, x=None, x_rows=1, index=A, nbytes=0), "x is NULL") == -1
    assert code(lib, ragged(lib, x=None, x_rows=0, nbytes=0), "no index") == -1


def test_a_type_that_contradicts_the_output_is_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = eg.Mx4Weight(torch.zeros(17408, dtype=torch.uint8), 0, 8, 64, 0, None)
    many = w._replace(sets=2, packed=torch.zeros(34816, dtype=torch.uint8))
    byte = torch.zeros(4, 32, dtype=torch.uint8)
    rows = eg.Mx4Rows(byte, byte[:, :2].contiguous(), torch.zeros(17408, dtype=torch.uint8), 4, 64,
                      0, None)
    off = torch.zeros(3, dtype=torch.int32)
    half, wide = torch.float16, torch.zeros(4, 64, dtype=torch.float16)
    y = wide[:, :8].contiguous()
    for call in (lambda d: eg.mx4_dequant(rows, dtype=d, out=wide),
                 lambda d: eg.mx4_gemm(rows, w, dtype=d, out=y),
                 lambda d: eg.mx4_linear(x, w, dtype=d, out=y),
                 lambda d: eg.mx4_linear_ragged(x, off, many, dtype=d, out=y)):
        for d in (torch.float32, torch.bfloat16):
            with pytest.raises(TypeError, match="dtype"):
                call(d)
        for d in (None, half):  # (as far as the device, which these tensors are not on)
            with pytest.raises(ValueError, match="CUDA"):
                call(d)


def test_what_is_written_lies_apart_from_what_is_read(lib):  # noqa: F811
    # 4 rows of 64: x 512 bytes, codes 128, scales 8, an operand of 17408; a weight of
    # 8 x 64: codes 256, scales 16, 17408 packed
    far = [2 * A, 3 * A, 4 * A]
    for at in range(3):
        for to in (A, A + 496, A - (112, 0, 17392)[at]):
            out = far[:at] + [to] + far[at + 1:]
            assert code(lib, q(lib, c=out[0], s=out[1], op=out[2]), "overlaps x") == -1, (at, to)
    d = lib.egopq_mx4_dequant
    for y in (A, A + 112, A - 496, 2 * A, 2 * A - 496):
        assert code(lib, d(A, 2 * A, 4, 64, 0, None, 0, y, None), "y overlaps") == -1
    for y in (A, A + 17392, 2 * A - 48, 2 * A + 17392):
        assert code(lib, lib.egopq_mx4_gemm(A, 2 * A, None, None, 4, 8, 64, 0, 0, y, None),
                    "y overlaps") == -1
    for p in (A - 17392, A + 240, 2 * A):
        assert code(lib, lib.egopq_mx4_pack(A, 2 * A, 1, 8, 64, 0, p, None), "overlaps") == -1
        assert code(lib, lib.egopq_mx4_unpack(p, 1, 8, 64, 0, A, 2 * A, None), "overlaps") == -1
    w = 8 * A
    assert code(lib, linear(lib, w=w, y=w + 17392), "overlaps packed") == -1
    assert code(lib, linear(lib, w=w, work=w - 17392), "overlaps packed") == -1
    for word in ("offsets", "index"):
        for at, what in ((2 * A + 60, "y"), (3 * A, "workspace")):
            k = {"off": 9 * A, "index": 10 * A, "off" if word == "offsets" else "index": at}
            assert code(lib, ragged(lib, **k), f"{what} overlaps {word}") == -1
