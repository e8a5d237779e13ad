"""Refusals and sizes of the operators whose weights each row picks (host
checks only: no device is touched)."""
import pytest
import torch

import w4a8_quantized_gemm_gb300 as eg
from w4a8_quantized_gemm_gb300 import builder

A = 0x10000  # an aligned address that is never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return eg.load()


def route(lib, logits=A, bf16=0, bias=None, T=4, E=64, k=6, score=0, groups=1, keep=1, gs=0,
          renorm=1, scale=1.0, weights=A, ids=A):
    return lib.egopq_moe_route(logits, bf16, bias, T, E, k, score, groups, keep, gs, renorm, scale,
                               weights, ids, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), -1), (dict(weights=None), -1), (dict(ids=None), -1),
    (dict(logits=A + 4), -3), (dict(bias=A + 8), -3), (dict(T=-1), -1), (dict(E=0), -1),
    (dict(k=0), -1), (dict(k=65), -1), (dict(score=2), -1), (dict(gs=2), -1),
    (dict(groups=0), -1), (dict(groups=5), -1), (dict(groups=8, keep=9), -1),
    (dict(groups=8, keep=0), -1), (dict(groups=16, keep=1, k=5), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(E=1024), -2),
    (dict(k=33), -2), (dict(groups=64, keep=64), -2), (dict(T=1 << 31), -2)])
def test_route_refusals(lib, kw, code):
    assert route(lib, **kw) == code
    assert lib.egopq_last_error_string()


def test_empty_batches_are_no_ops(lib):
    assert route(lib, T=0, logits=None, weights=None, ids=None) == 0
    assert lib.egopq_moe_experts(None, None, None, None, None, 0, 2, 8, 256, 256, 128, 0, None,
                                 None, 0, 0, None) == 0
    assert lib.egopq_lora_add(None, None, None, None, None, None, None, 0, 256, 256, 4, 16, None,
                              None, 0, None) == 0
    assert lib.egopq_w4a8_linear_lora(None, None, None, None, None, None, None, 0, 256, 256, 128,
                                      4, 16, None, None, 0, 0, None) == 0


def experts(lib, x=A, ids=A, w=A, gu=A, dn=A, T=4, k=2, E=8, H=256, I=256, group=128, variant=0,
            out=A, ws=A, nbytes=1 << 40, path=0):
    return lib.egopq_moe_experts(x, ids, w, gu, dn, T, k, E, H, I, group, variant, out, ws, nbytes,
                                 path, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(ids=None), -1), (dict(w=None), -1), (dict(gu=None), -1),
    (dict(dn=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(x=A + 2), -3),
    (dict(ws=A + 8), -3), (dict(T=-1), -1), (dict(k=0), -1), (dict(E=0), -1), (dict(H=200), -2),
    (dict(I=64), -2), (dict(group=64), -2), (dict(variant=2), -1), (dict(variant=7), -1),
    (dict(E=1025), -2), (dict(T=1 << 31), -2), (dict(T=1 << 30, k=4), -2), (dict(H=1 << 20), -2),
    (dict(path=3), -1), (dict(nbytes=100), -1)])
def test_experts_refusals(lib, kw, code):
    assert experts(lib, **kw) == code
    assert lib.egopq_last_error_string()


def lora(lib, y=A, x=A, a=A, b=A, s=A, ranks=None, ids=A, M=4, N=256, K=256, L=4, r=16, out=A, ws=A,
         nbytes=1 << 40):
    return lib.egopq_lora_add(y, x, a, b, s, ranks, ids, M, N, K, L, r, out, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), -1), (dict(x=None), -1), (dict(a=None), -1), (dict(b=None), -1),
    (dict(s=None), -1), (dict(ids=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(ranks=A + 4), -3), (dict(b=A + 8), -3), (dict(M=-1), -1), (dict(L=0), -1),
    (dict(r=0), -1), (dict(r=12), -2), (dict(r=136), -2), (dict(K=192), -2), (dict(N=100), -2),
    (dict(L=1025), -2), (dict(M=1 << 31), -2), (dict(N=1 << 24), -2), (dict(nbytes=64), -1)])
def test_lora_refusals(lib, kw, code):
    assert lora(lib, **kw) == code
    assert lib.egopq_last_error_string()


def test_linear_lora_checks_both_halves_before_a_launch(lib):
    def call(M=4, N=256, K=256, group=128, r=16, path=0, nbytes=1 << 40, ids=A):
        return lib.egopq_w4a8_linear_lora(A, A, A, A, A, None, ids, M, N, K, group, 4, r, A, A,
                                          nbytes, path, None)
    assert call(group=64) == -2
    assert call(r=12) == -2
    assert call(path=5) == -1
    assert call(nbytes=1000) == -1
    assert call(ids=None) == -1


def test_workspace_sizes(lib):
    ws = lib.egopq_moe_experts_workspace_bytes
    assert ws(0, 2, 8, 256, 256, 128, 0, 0) == 0
    assert ws(4, 2, 8, 200, 256, 128, 0, 0) == 0
    sizes = [ws(T, 4, 16, 512, 256, 128, 0, 0) for T in (1, 3, 16, 17, 100, 513, 4096)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert lib.egopq_lora_workspace_bytes(1, 256, 256, 4, 16) > 0
    assert lib.egopq_lora_workspace_bytes(1, 256, 256, 4, 12) == 0
    assert lib.egopq_w4a8_linear_lora_workspace_bytes(8, 256, 256, 64, 4, 16, 0) == 0


def test_binding_checks_shapes_and_types():
    t = torch.zeros
    with pytest.raises(TypeError):
        eg.moe_route(t(2, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        eg.moe_route(t(2, 8), 2, bias=t(7))
    with pytest.raises(ValueError):
        eg.LoraAdapters(t(2, 8, 128, dtype=torch.bfloat16), t(2, 128, 16, dtype=torch.bfloat16),
                        t(2))
    with pytest.raises(ValueError):
        eg.LoraAdapters(t(2, 8, 128, dtype=torch.bfloat16), t(2, 128, 8, dtype=torch.bfloat16),
                        t(3))
