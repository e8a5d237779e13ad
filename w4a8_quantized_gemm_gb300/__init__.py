"""GB300 (sm_103a) W4A8 packed-linear GEMM: thin Python binding of libegopq.

Argument marshalling only: every step of the path runs in the CUDA kernels of
`libegopq.so` (built in-tree by `w4a8_quantized_gemm_gb300.builder`). PyTorch
provides device memory and the current stream. There is no CPU fallback: if the
library is missing or the device is not sm_103, calls raise.

Typical use (one linear, W4A8):

    packed = pack_w4(w_q, scale_f16, zero)            # once per weight
    a = quant_act(x)                                  # per token batch
    y = w4a8_gemm(a, packed, N, K)                    # bf16 [M, N]

A call runs on the current stream, or on `stream`; the tensors it is given have
to be ready there. What it allocates itself is `stream`'s memory (as under
torch.cuda.stream(stream)), and the caller's stream may read its results once it
has waited for `stream`.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libegopq.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "egopq.h")

PATH_AUTO, PATH_GEMV, PATH_TC = 0, 1, 2
VARIANT_W4A8, VARIANT_W4A16, VARIANT_W8A16, VARIANT_W8A8 = 0, 1, 2, 3
STATUS = {0: "OK", -1: "INVALID_ARG", -2: "UNSUPPORTED_SHAPE", -3: "MISALIGNED",
          -4: "ARCH", -5: "CUDA", -6: "TIMEOUT", -7: "DEVICE_INDEX"}
DEBUG_LIB_PATH = os.path.join(_HERE, "_build", "libegopq_debug.so")
GROUP = 128

_lock = threading.Lock()
_lib = None


class EgopqError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"egopq error {code} ({STATUS.get(code, '?')}): {msg}")
        self.code = code


def build(force: bool = False) -> str:
    from . import builder
    return builder.build(force=force)


def load() -> ctypes.CDLL:
    """Load libegopq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m w4a8_quantized_gemm_gb300.builder`")
        lib = ctypes.CDLL(LIB_PATH)
        i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        sig = {
            "egopq_version": (i32, []),
            "egopq_last_error_string": (ctypes.c_char_p, []),
            "egopq_packed_w4_bytes": (sz, [i64, i64, i32]),
            "egopq_pack_w4": (i32, [vp, vp, vp, i64, i64, i32, vp, vp]),
            "egopq_unpack_w4": (i32, [vp, i64, i64, i32, vp, vp, vp, vp]),
            "egopq_dequant_w4": (i32, [vp, i64, i64, i32, vp, vp]),
            "egopq_pack_w4_gptq": (i32, [vp, vp, vp, i64, i64, i32, i32, vp, vp]),
            "egopq_quant_act_i8": (i32, [vp, i64, i64, i32, vp, vp, vp, vp, vp]),
            "egopq_w4a8_gemm": (i32, [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, vp]),
            "egopq_w4a8_gemm_ex": (i32, [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32, vp]),
            "egopq_w4a8_group_partials": (i32, [vp, vp, vp, vp, i64, i64, i64, i32, vp, i32, vp]),
            "egopq_w4a16_gemm": (i32, [vp, vp, i64, i64, i64, i32, vp, vp]),
            "egopq_w4a16_gemm_ex": (i32, [vp, vp, i64, i64, i64, i32, vp, i32, vp]),
            "egopq_w8a16_gemm": (i32, [vp, vp, vp, i64, i64, i64, vp, vp]),
            "egopq_w8a16_gemm_ex": (i32, [vp, vp, vp, i64, i64, i64, vp, i32, vp]),
            "egopq_w8a8_gemm": (i32, [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]),
            "egopq_w8a8_gemm_ex": (i32, [vp, vp, vp, vp, vp, i64, i64, i64, vp, i32, vp]),
            "egopq_w4a8_linear_workspace_bytes": (sz, [i64, i64, i32, i32]),
            "egopq_w4a8_linear": (i32, [vp, vp, i64, i64, i64, i32, vp, vp, sz, i32, vp]),
            "egopq_w4a8_linear_noalloc": (i32, [vp, vp, i64, i64, i64, i32, vp, i32, vp]),
            "egopq_w4a8_gemm_grouped": (i32, [vp, vp, vp, vp, i32, vp, vp, i64, i64, i32, vp,
                                              i32, vp]),
            "egopq_w4a8_linear_grouped": (i32, [vp, i32, vp, vp, i64, i64, i32, vp, vp, sz, i32,
                                                vp]),
            "egopq_bf16_gemm_twin": (i32, [vp, vp, i64, i64, i64, vp, vp]),
            "egopq_moe_route": (i32, [vp, i32, vp, i64, i32, i32, i32, i32, i32, i32, i32,
                                      ctypes.c_float, vp, vp, vp]),
            "egopq_moe_pack_gate_up": (i32, [vp, vp, vp, i64, i64, i64, i32, vp, vp]),
            "egopq_moe_experts_workspace_bytes": (sz, [i64, i32, i32, i64, i64, i32, i32, i32]),
            "egopq_moe_experts": (i32, [vp, vp, vp, vp, vp, i64, i32, i32, i64, i64, i32, i32, vp,
                                        vp, sz, i32, vp]),
            "egopq_lora_workspace_bytes": (sz, [i64, i64, i64, i32, i32]),
            "egopq_lora_add": (i32, [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, vp,
                                     sz, vp]),
            "egopq_w4a8_linear_lora_workspace_bytes": (sz, [i64, i64, i64, i32, i32, i32, i32]),
            "egopq_w4a8_linear_lora": (i32, [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32,
                                             i32, vp, vp, sz, i32, vp]),
            "egopq_mx4_operand_bytes": (sz, [i64, i64, i32]),
            "egopq_mx4_quant": (i32, [vp, i32, i64, i64, i32, vp, i32, vp, vp, vp, vp]),
            "egopq_mx4_dequant": (i32, [vp, vp, i64, i64, i32, vp, i32, vp, vp]),
            "egopq_mx4_packed_bytes": (sz, [i64, i64, i64, i32]),
            "egopq_mx4_pack": (i32, [vp, vp, i64, i64, i64, i32, vp, vp]),
            "egopq_mx4_unpack": (i32, [vp, i64, i64, i64, i32, vp, vp, vp]),
            "egopq_mx4_gemm": (i32, [vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, vp]),
            "egopq_mx4_linear_workspace_bytes": (sz, [i64, i64, i64, i32]),
            "egopq_mx4_linear": (i32, [vp, i32, i64, i64, i64, i32, vp, vp, vp, i32, i32, vp, vp,
                                       sz, vp]),
            "egopq_mx4_linear_ragged": (i32, [vp, i32, i64, vp, vp, i64, i64, i64, i64, i32, vp,
                                              vp, vp, i32, i32, vp, vp, sz, vp]),
            "egopq_supported": (i32, [i64, i64, i64, i32, i32]),
            "egopq_auto_path": (i32, [i64, i32]),
            "egopq_tc_operand_bytes": (sz, [i64, i64, i32]),
            "egopq_tc_operand_form": (i32, [i64]),
            "egopq_tc_token_tile": (i32, [i64, i64, i64, i32]),
            "egopq_tc_launches": (i32, [i64, i64, i64, i32]),
            "egopq_device_status": (i32, [vp]),
            "egopq_selftest_timeout": (i32, [i32, vp]),
            "egopq_debug_build": (i32, []),
            "egopq_debug_set_record_limit": (i32, [ctypes.c_uint64]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def header_functions() -> list:
    """Names of the functions include/egopq.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(egopq_[a-z0-9_]+)\s*\(", text)))


# ------------------------------------------------------------------ helpers --

def _check(rc: int):
    if rc != 0:
        raise EgopqError(rc, load().egopq_last_error_string().decode(errors="replace"))


def _stream(stream: Optional[torch.cuda.Stream] = None) -> int:
    if stream is None:  # (the raw handle: a Stream object a call costs microseconds)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _scratch(shape, dtype: torch.dtype, device, stream=None) -> torch.Tensor:
    """Memory for a call's kernels. Where a stream is given it is that stream's,
    as under torch.cuda.stream(stream): what had the memory before, and what gets
    it next, is then in order with those kernels without any event."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _output(shape, dtype: torch.dtype, device, stream=None) -> torch.Tensor:
    """A result a call allocates: as _scratch, and not given out again before
    the caller's own stream, which may read it, has come as far as where the
    caller lets go of it."""
    t = _scratch(shape, dtype, device, stream)
    if stream is not None:
        here = torch.cuda.current_stream(device)
        if here != stream:
            t.record_stream(here)
    return t


def _dtype(t: torch.Tensor, *dtypes):
    if t.dtype not in dtypes:  # (dtypes are compared by identity)
        raise TypeError(f"expected dtype in {dtypes}, got {t.dtype}")


# --------------------------------------------------------------------- API ---

def packed_w4_bytes(N: int, K: int, group: int = GROUP) -> int:
    return int(load().egopq_packed_w4_bytes(N, K, group))


def pack_w4(w_q: torch.Tensor, scale_f16: torch.Tensor, zero: torch.Tensor,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """w_q uint8 [N,K] codes 0..15, scale fp16 [N,G], zero uint8 [N,G] -> packed uint8."""
    _dtype(w_q, torch.uint8)
    _dtype(scale_f16, torch.float16, torch.int16, torch.uint16)
    _dtype(zero, torch.uint8)
    N, K = w_q.shape
    nbytes = packed_w4_bytes(N, K)
    if nbytes == 0:
        raise EgopqError(-2, f"shape N={N} K={K} is not packable (K, N multiples of 128)")
    if out is None:
        out = _output(nbytes, torch.uint8, w_q.device, stream)
    _check(load().egopq_pack_w4(_ptr(w_q), _ptr(scale_f16), _ptr(zero), N, K, GROUP,
                                _ptr(out), _stream(stream)))
    return out


def unpack_w4(packed: torch.Tensor, N: int, K: int, stream=None):
    G = K // GROUP
    dev = packed.device
    w = _output((N, K), torch.uint8, dev, stream)
    s = _output((N, G), torch.float16, dev, stream)
    z = _output((N, G), torch.uint8, dev, stream)
    _check(load().egopq_unpack_w4(_ptr(packed), N, K, GROUP, _ptr(w), _ptr(s), _ptr(z),
                                  _stream(stream)))
    return w, s, z


def pack_w4_gptq(qweight: torch.Tensor, qzeros: torch.Tensor, scales: torch.Tensor,
                 zero_offset: int = 1, stream=None) -> torch.Tensor:
    """Packed weight from a GPTQ checkpoint's qweight int32 [K/8, N], qzeros
    int32 [G, N/8] and scales fp16 [G, N] (layout in include/egopq.h)."""
    _dtype(qweight, torch.int32)
    _dtype(qzeros, torch.int32)
    K, N = qweight.shape[0] * 8, qweight.shape[1]
    packed = _output(packed_w4_bytes(N, K), torch.uint8, qweight.device, stream)
    _check(load().egopq_pack_w4_gptq(_ptr(qweight), _ptr(qzeros), _ptr(scales), N, K, GROUP,
                                     zero_offset, _ptr(packed), _stream(stream)))
    return packed


def dequant_w4(packed: torch.Tensor, N: int, K: int, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """The packed weight dequantized once to dense bf16 [N, K]."""
    if out is None:
        out = _output((N, K), torch.bfloat16, packed.device, stream)
    _check(load().egopq_dequant_w4(_ptr(packed), N, K, GROUP, _ptr(out), _stream(stream)))
    return out


class QuantAct(NamedTuple):
    # int8 [M, K], or None when the codes were written only in the tensor-core
    # operand form (all the tensor-core path reads)
    a_q: Optional[torch.Tensor]
    a_s: torch.Tensor      # fp32 [M]
    a_gsum: torch.Tensor   # int32 [M, G]
    # uint8: the codes in the tensor-core operand form the library picks for
    # this M (tc_operand_form; layout in include/egopq.h), or None
    a_tc: Optional[torch.Tensor]


TC_FORM_E4M3_PLANES, TC_FORM_F16 = 1, 2


def auto_path(M: int, variant: int = VARIANT_W4A8) -> int:
    """The path (PATH_GEMV or PATH_TC) the library's AUTO choice takes for M
    tokens of `variant`."""
    rc = int(load().egopq_auto_path(M, variant))
    if rc < 0:
        _check(rc)
    return rc


def tc_token_tile(M: int, N: int, K: int, variant: int = VARIANT_W4A8) -> int:
    """Tokens per output tile (the MMA's N) the tensor-core path runs an
    M x N x K call of `variant` with on the current device."""
    rc = int(load().egopq_tc_token_tile(M, N, K, variant))
    if rc < 0:
        _check(rc)
    return rc


def tc_launches(M: int, N: int, K: int, variant: int = VARIANT_W4A8) -> int:
    """Kernel launches (1 or 2) the tensor-core path makes for an M x N x K
    call of `variant` on the current device."""
    rc = int(load().egopq_tc_launches(M, N, K, variant))
    if rc < 0:
        _check(rc)
    return rc


def tc_operand_form(M: int) -> int:
    """TC_FORM_E4M3_PLANES or TC_FORM_F16: the form quant_act writes the
    tensor-core operand in for M tokens."""
    rc = int(load().egopq_tc_operand_form(M))
    if rc < 0:
        _check(rc)
    return rc


def tc_operand(M: int, K: int, device, stream=None) -> torch.Tensor:
    """A buffer for the tensor-core operand form of M x K codes (empty for an
    empty batch)."""
    if M == 0:
        return _output((0,), torch.uint8, device, stream)
    nbytes = int(load().egopq_tc_operand_bytes(M, K, GROUP))
    if nbytes == 0:
        raise EgopqError(-2, f"no tensor-core operand for M={M} K={K}")
    return _output((nbytes,), torch.uint8, device, stream)


def quant_act(x: torch.Tensor, with_tc: bool = True, out: Optional[QuantAct] = None,
              stream=None, with_codes: bool = True) -> QuantAct:
    """Per-token symmetric int8 quantization of bf16 x [M, K]. with_codes=False
    leaves the int8 codes out (a_q None): only the tensor-core path can read
    the result."""
    _dtype(x, torch.bfloat16, torch.int16, torch.uint16)
    M, K = x.shape
    if out is None:
        dev = x.device
        out = QuantAct(_output((M, K), torch.int8, dev, stream) if with_codes else None,
                       _output((M,), torch.float32, dev, stream),
                       _output((M, max(K // GROUP, 1)), torch.int32, dev, stream),
                       tc_operand(M, K, dev, stream) if with_tc else None)
    _check(load().egopq_quant_act_i8(_ptr(x), M, K, GROUP, _ptr(out.a_q), _ptr(out.a_s),
                                     _ptr(out.a_gsum), _ptr(out.a_tc), _stream(stream)))
    return out


def w4a8_gemm(a: QuantAct, packed: torch.Tensor, N: int, K: int, path: int = PATH_AUTO,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    M = a.a_s.shape[0]
    if out is None:
        out = _output((M, N), torch.bfloat16, a.a_s.device, stream)
    _check(load().egopq_w4a8_gemm_ex(_ptr(a.a_q), _ptr(a.a_tc), _ptr(a.a_s), _ptr(a.a_gsum),
                                     _ptr(packed), M, N, K, GROUP, _ptr(out), path,
                                     _stream(stream)))
    return out


def w4a8_linear_workspace_bytes(M: int, K: int, path: int = PATH_AUTO) -> int:
    return int(load().egopq_w4a8_linear_workspace_bytes(M, K, GROUP, path))


def w4a8_linear(x: torch.Tensor, packed: torch.Tensor, N: int, path: int = PATH_AUTO,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """One-call W4A8 linear from bf16 x [M, K]: per-token int8 quantization into
    a workspace, then the W4A8 GEMM (two kernels, one call)."""
    _dtype(x, torch.bfloat16)
    M, K = x.shape
    if out is None:
        out = _output((M, N), torch.bfloat16, x.device, stream)
    need = w4a8_linear_workspace_bytes(M, K, path)
    if workspace is None:
        workspace = _scratch(need, torch.uint8, x.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().egopq_w4a8_linear(_ptr(x), _ptr(packed), M, N, K, GROUP, _ptr(out),
                                    _ptr(workspace), ws_bytes, path, _stream(stream)))
    return out


class _Group:
    """Host arrays (packed pointers, row counts, output pointers) of sibling
    linears for the grouped calls; built once, reused by every call."""

    def __init__(self, packed, N, outs):
        n = len(packed)
        if not (1 <= n <= 8) or len(N) != n or len(outs) != n:
            raise ValueError("1 to 8 linears, with one N and one output each")
        self.count = n
        self.packed = (ctypes.c_void_p * n)(*[_ptr(p) for p in packed])
        self.N = (ctypes.c_int64 * n)(*[int(v) for v in N])
        self.y = (ctypes.c_void_p * n)(*[_ptr(o) for o in outs])


def _grouped_outputs(M, N, device, out, stream):
    if out is None:
        out = [_output((M, n), torch.bfloat16, device, stream) for n in N]
    for o, n in zip(out, N):
        _dtype(o, torch.bfloat16)
        if tuple(o.shape) != (M, n):
            raise ValueError(f"output of shape {tuple(o.shape)}, expected {(M, n)}")
    return out


def w4a8_gemm_grouped(a: QuantAct, packed: list, N: list, K: int, path: int = PATH_AUTO,
                      out: Optional[list] = None, stream=None) -> list:
    """Sibling linears sharing the activations `a` (q|k|v, gate|up) in one
    launch: returns [y_j bf16 [M, N_j]]."""
    M = a.a_s.shape[0]
    out = _grouped_outputs(M, N, a.a_s.device, out, stream)
    g = _Group(packed, N, out)
    _check(load().egopq_w4a8_gemm_grouped(_ptr(a.a_q), _ptr(a.a_tc), _ptr(a.a_s), _ptr(a.a_gsum),
                                          g.count, g.packed, g.N, M, K, GROUP, g.y, path,
                                          _stream(stream)))
    return out


def w4a8_linear_grouped(x: torch.Tensor, packed: list, N: list, path: int = PATH_AUTO,
                        out: Optional[list] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> list:
    """One quantization of bf16 x [M, K] and one grouped GEMM over the sibling
    weights: returns [y_j bf16 [M, N_j]]."""
    _dtype(x, torch.bfloat16)
    M, K = x.shape
    out = _grouped_outputs(M, N, x.device, out, stream)
    need = w4a8_linear_workspace_bytes(M, K, path)
    if workspace is None:
        workspace = _scratch(need, torch.uint8, x.device, stream)
    g = _Group(packed, N, out)
    _check(load().egopq_w4a8_linear_grouped(_ptr(x), g.count, g.packed, g.N, M, K, GROUP, g.y,
                                            _ptr(workspace), workspace.numel(), path,
                                            _stream(stream)))
    return out


def w4a8_group_partials(a: QuantAct, packed: torch.Tensor, N: int, K: int,
                        path: int = PATH_TC, stream=None) -> torch.Tensor:
    M = a.a_s.shape[0]
    Q = _output((M, N, K // GROUP), torch.int32, a.a_s.device, stream)
    _check(load().egopq_w4a8_group_partials(_ptr(a.a_q), _ptr(a.a_tc), _ptr(a.a_gsum),
                                            _ptr(packed), M, N, K, GROUP, _ptr(Q), path,
                                            _stream(stream)))
    return Q


def w4a16_gemm(x: torch.Tensor, packed: torch.Tensor, N: int, K: int, path: int = PATH_AUTO,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _dtype(x, torch.bfloat16)
    M = x.shape[0]
    if out is None:
        out = _output((M, N), torch.bfloat16, x.device, stream)
    _check(load().egopq_w4a16_gemm_ex(_ptr(x), _ptr(packed), M, N, K, GROUP, _ptr(out), path,
                                      _stream(stream)))
    return out


def w8a16_gemm(x: torch.Tensor, w_q: torch.Tensor, scale_f16: torch.Tensor,
               path: int = PATH_AUTO, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    _dtype(x, torch.bfloat16)
    _dtype(w_q, torch.int8)
    M, K = x.shape
    N = w_q.shape[0]
    if out is None:
        out = _output((M, N), torch.bfloat16, x.device, stream)
    _check(load().egopq_w8a16_gemm_ex(_ptr(x), _ptr(w_q), _ptr(scale_f16), M, N, K, _ptr(out),
                                      path, _stream(stream)))
    return out


def w8a8_gemm(a: QuantAct, w_q: torch.Tensor, scale_f16: torch.Tensor, path: int = PATH_AUTO,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """W8A8 int8-dynamic GEMM: per-token int8 activations (from quant_act; a_tc
    is read on the tensor-core path only) times int8 weights [N, K] with fp16
    per-channel scales [N]."""
    _dtype(w_q, torch.int8)
    M = a.a_s.shape[0]
    N, K = w_q.shape
    if out is None:
        out = _output((M, N), torch.bfloat16, a.a_s.device, stream)
    _check(load().egopq_w8a8_gemm_ex(_ptr(a.a_q), _ptr(a.a_tc), _ptr(a.a_s), _ptr(w_q),
                                     _ptr(scale_f16), M, N, K, _ptr(out), path,
                                     _stream(stream)))
    return out


def bf16_gemm_twin(x: torch.Tensor, w: torch.Tensor, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Dense bf16 x [M, K] times w [N, K] through the W4A16 tensor-core
    pipeline with a copy in place of the int4 unpack (comparison kernel)."""
    _dtype(x, torch.bfloat16)
    _dtype(w, torch.bfloat16)
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = _output((M, N), torch.bfloat16, x.device, stream)
    _check(load().egopq_bf16_gemm_twin(_ptr(x), _ptr(w), M, N, K, _ptr(out), _stream(stream)))
    return out


# ------------------------------------------ rows that pick their own weights ---

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


def _shape(t: torch.Tensor, *shape):
    if t.shape != shape:
        raise ValueError(f"tensor of shape {tuple(t.shape)}, expected {shape}")


def _arg(t: torch.Tensor, dtype: torch.dtype, *shape) -> int:
    """The device address of a tensor of this type and shape, after the checks
    every call makes (in one test: they are on the path of single tokens)."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _dtype(t, dtype)
    _shape(t, *shape)
    return _ptr(t)


def moe_route(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None,
              score: int = SCORE_SOFTMAX, n_group: int = 1, topk_group: int = 1,
              group_score: int = GROUP_MAX, renorm: bool = True, scale: float = 1.0,
              out: Optional[tuple] = None, stream=None) -> tuple:
    """The k experts of each token and their weights from router logits [T, E]
    (fp32 or bf16): returns (weights fp32 [T, k], ids int32 [T, k]), the best
    expert first (include/egopq.h has the formulas)."""
    bf16 = logits.dtype is torch.bfloat16
    if not bf16:
        _dtype(logits, torch.float32, torch.bfloat16)
    T, E = logits.shape
    if out is None:
        out = (_output((T, k), torch.float32, logits.device, stream),
               _output((T, k), torch.int32, logits.device, stream))
    weights, ids = out
    _check(load().egopq_moe_route(
        _arg(logits, logits.dtype, T, E), bf16,
        None if bias is None else _arg(bias, torch.float32, E), T, E, k, score, n_group,
        topk_group, group_score, renorm, scale, _arg(weights, torch.float32, T, k),
        _arg(ids, torch.int32, T, k), _stream(stream)))
    return out


class MoeLayer(NamedTuple):
    """Packed weights of a layer's experts (moe_pack)."""
    gate_up: torch.Tensor  # uint8, gate and up rows interleaved
    down: torch.Tensor     # uint8
    E: int
    H: int
    I: int


def moe_pack(gate_up_q: torch.Tensor, gate_up_scale: torch.Tensor, gate_up_zero: torch.Tensor,
             down_q: torch.Tensor, down_scale: torch.Tensor, down_zero: torch.Tensor,
             stream=None) -> MoeLayer:
    """Pack the experts of a layer: gate_up uint8 codes [E, 2I, H] (I gate rows,
    then I up rows) with fp16 scales and uint8 zero points [E, 2I, H/128], and
    down codes [E, H, I] with theirs [E, H, I/128]."""
    E, I2, H = gate_up_q.shape
    I = I2 // 2
    if I2 % 2:
        raise ValueError(f"{I2} gate and up rows: an odd number")
    nbytes = packed_w4_bytes(E * I2, H)
    if nbytes == 0 or I % GROUP:
        raise EgopqError(-2, f"experts with H={H} I={I} are not packable (multiples of 128)")
    q, s, z = (_arg(gate_up_q, torch.uint8, E, I2, H),
               _arg(gate_up_scale, torch.float16, E, I2, H // GROUP),
               _arg(gate_up_zero, torch.uint8, E, I2, H // GROUP))
    for t, dtype, K in ((down_q, torch.uint8, I), (down_scale, torch.float16, I // GROUP),
                        (down_zero, torch.uint8, I // GROUP)):
        _arg(t, dtype, E, H, K)
    packed = _output(nbytes, torch.uint8, gate_up_q.device, stream)
    _check(load().egopq_moe_pack_gate_up(q, s, z, E, I, H, GROUP, packed.data_ptr(),
                                         _stream(stream)))
    down = pack_w4(down_q.view(E * H, I), down_scale.view(E * H, I // GROUP),
                   down_zero.view(E * H, I // GROUP), stream=stream)
    return MoeLayer(packed, down, E, H, I)


def moe_workspace_bytes(T: int, k: int, E: int, H: int, I: int, variant: int = VARIANT_W4A8,
                        path: int = PATH_AUTO) -> int:
    return int(load().egopq_moe_experts_workspace_bytes(T, k, E, H, I, GROUP, variant, path))


def moe_workspace(T: int, k: int, E: int, H: int, I: int, variant: int, device,
                  path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """A workspace for moe_experts of T tokens (and of any fewer), of the stream
    it is to be used on."""
    return _scratch(moe_workspace_bytes(T, k, E, H, I, variant, path), torch.uint8, device, stream)


def moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, layer: MoeLayer,
                variant: int = VARIANT_W4A8, path: int = PATH_AUTO,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """The gated linears of the experts each token picked, summed with its
    weights: x bf16 [T, H], ids int32 and weights fp32 [T, k] -> bf16 [T, H].
    An id outside [0, E) adds nothing."""
    gate_up, down, E, H, I = layer
    T, k = ids.shape
    if out is None:
        out = _output((T, H), torch.bfloat16, x.device, stream)
    if workspace is None:
        workspace = moe_workspace(T, k, E, H, I, variant, x.device, path, stream)
    _check(load().egopq_moe_experts(
        _arg(x, torch.bfloat16, T, H), _arg(ids, torch.int32, T, k),
        _arg(weights, torch.float32, T, k), gate_up.data_ptr(), down.data_ptr(), T, k, E, H, I,
        GROUP, variant, _arg(out, torch.bfloat16, T, H), _ptr(workspace), workspace.nbytes, path,
        _stream(stream)))
    return out


class LoraAdapters:
    """The low-rank adapters of one projection: A bf16 [L, r, K], B bf16
    [L, N, r], scale fp32 [L], ranks int32 [L] (adapter a uses its first
    ranks[a]; None: r everywhere). The tensors stay as they are named; their
    values may change, and so may the memory behind them (t.data = ..., resize_):
    each call reads their addresses, and one that moved is checked again. Until
    then the memory that was checked is kept."""

    __slots__ = ("A", "B", "scale", "ranks", "L", "r", "K", "N", "_ptrs", "_kept")

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                 ranks: Optional[torch.Tensor] = None):
        L, r, K = A.shape
        N = B.shape[1]
        for name, v in zip(self.__slots__, (A, B, scale, ranks, L, r, K, N)):
            object.__setattr__(self, name, v)
        self._check()

    def __setattr__(self, name, value):
        raise AttributeError(f"LoraAdapters.{name} is fixed: make new adapters")

    def _check(self):
        L, r, K, N = self.L, self.r, self.K, self.N
        tensors = (self.A, self.B, self.scale, self.ranks)
        for t, dtype, shape in zip(tensors, (torch.bfloat16, torch.bfloat16, torch.float32,
                                             torch.int32),
                                   ((L, r, K), (L, N, r), (L,), (L,))):
            if t is not None:
                _dtype(t, dtype)
                _shape(t, *shape)
        object.__setattr__(self, "_ptrs", tuple(_ptr(t) for t in tensors))
        # an address that is still the same is then still this memory
        object.__setattr__(self, "_kept", tuple(t.untyped_storage() for t in tensors
                                                if t is not None))

    def _addresses(self) -> tuple:
        """Where A, B, scale and ranks lie now."""
        ranks = self.ranks
        ptrs = (self.A.data_ptr(), self.B.data_ptr(), self.scale.data_ptr(),
                None if ranks is None else ranks.data_ptr())
        if ptrs != self._ptrs:
            self._check()
        return ptrs


def lora_workspace(M: int, N: int, K: int, adapters: LoraAdapters, device,
                   stream=None) -> torch.Tensor:
    """A workspace for lora_add of M rows (and of any fewer), of the stream it is
    to be used on."""
    return _scratch(int(load().egopq_lora_workspace_bytes(M, N, K, adapters.L, adapters.r)),
                    torch.uint8, device, stream)


def lora_add(y: torch.Tensor, x: torch.Tensor, adapters: LoraAdapters, ids: torch.Tensor,
             workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """y [M, N] + scale * B_a (A_a x[m]) for each row's adapter a = ids[m] (rows
    with an id outside [0, L) keep y); bf16. `out` may be y itself."""
    A, B, scale, ranks = adapters._addresses()
    L, r, K, N = adapters.L, adapters.r, adapters.K, adapters.N
    M = x.shape[0]
    if out is None:
        out = _output((M, N), torch.bfloat16, x.device, stream)
    if workspace is None:
        workspace = lora_workspace(M, N, K, adapters, x.device, stream)
    _check(load().egopq_lora_add(
        _arg(y, torch.bfloat16, M, N), _arg(x, torch.bfloat16, M, K), A, B, scale, ranks,
        _arg(ids, torch.int32, M), M, N, K, L, r,
        _arg(out, torch.bfloat16, M, N), _ptr(workspace), workspace.nbytes, _stream(stream)))
    return out


def w4a8_linear_lora_workspace(M: int, N: int, K: int, adapters: LoraAdapters, device,
                               path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """A workspace for w4a8_linear_lora of M rows (and of any fewer), of the
    stream it is to be used on."""
    n = int(load().egopq_w4a8_linear_lora_workspace_bytes(M, N, K, GROUP, adapters.L, adapters.r,
                                                          path))
    return _scratch(n, torch.uint8, device, stream)


def w4a8_linear_lora(x: torch.Tensor, packed: torch.Tensor, N: int, adapters: LoraAdapters,
                     ids: torch.Tensor, path: int = PATH_AUTO,
                     workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """w4a8_linear of x [M, K] and the adapters' update of its output, in one
    call."""
    A, B, scale, ranks = adapters._addresses()
    L, r, K = adapters.L, adapters.r, adapters.K
    M = x.shape[0]
    if N != adapters.N:
        raise ValueError(f"adapters of {adapters.N} outputs beside a projection of {N}")
    if out is None:
        out = _output((M, N), torch.bfloat16, x.device, stream)
    if workspace is None:
        workspace = w4a8_linear_lora_workspace(M, N, K, adapters, x.device, path, stream)
    _check(load().egopq_w4a8_linear_lora(
        _arg(x, torch.bfloat16, M, K), _ptr(packed), A, B, scale, ranks,
        _arg(ids, torch.int32, M), M, N, K, GROUP, L, r, _arg(out, torch.bfloat16, M, N),
        _ptr(workspace), workspace.nbytes, path, _stream(stream)))
    return out


# --------------------------------------------------- microscaled 4-bit linears ---

MX4_E8M0, MX4_E4M3 = 0, 1
_MX4_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


_MX4_BLOCK = {MX4_E8M0: 32, MX4_E4M3: 16}


def mx4_block(fmt: int) -> int:
    """Neighbours along K that share a scale: 32 (MX4_E8M0) or 16 (MX4_E4M3)."""
    block = _MX4_BLOCK.get(fmt)
    if block is None:
        raise ValueError(f"unknown 4-bit format {fmt}")
    return block


def _mx4_here(first: torch.Tensor, *others) -> int:
    """The current device, which the kernels run on: a tensor of another, or of
    none, is refused (None is not)."""
    if not first.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    device = torch._C._cuda_getDevice()
    for t in (first, *others):
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensor on {t.device}, the current device is {device}")
    return device


def _mx4_at(t: torch.Tensor) -> int:
    """The address of a tensor that is on the device."""
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _mx4_stream(stream, device: int) -> int:
    return (torch._C._cuda_getCurrentRawStream(device) if stream is None
            else stream.cuda_stream)


def _mx4_type(dtype: torch.dtype) -> int:
    t = _MX4_TYPES.get(dtype)
    if t is None:
        raise TypeError(f"expected dtype in {tuple(_MX4_TYPES)}, got {dtype}")
    return t


def _mx4_result(dtype: Optional[torch.dtype], out: Optional[torch.Tensor],
                default: torch.dtype) -> torch.dtype:
    """The type of a result: that of `out`, which dtype may not contradict."""
    if out is None:
        return dtype or default
    if dtype is not None and dtype is not out.dtype:
        raise TypeError(f"dtype {dtype} for an out of {out.dtype}")
    return out.dtype


def _mx4_scale(t: Optional[torch.Tensor], n: int) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is torch.float32 and t.shape == (n,) and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _arg(t.reshape(1) if n == 1 and t.dim() == 0 else t, torch.float32, n)


class Mx4Rows(NamedTuple):
    """Rows in 4 bits (mx4_quant): codes uint8 [M, K/2] and scales uint8
    [M, K/block], or None; the form the products read, or None; the tensor's
    scale (MX4_E4M3), or None for 1."""
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    a_tc: Optional[torch.Tensor]
    M: int
    K: int
    fmt: int
    tensor_scale: Optional[torch.Tensor]


class Mx4Weight(NamedTuple):
    """A packed 4-bit weight, or the weights of `sets` experts (mx4_pack). One weight's
    `packed` may also be the a_tc of an mx4_quant of its N rows."""
    packed: torch.Tensor
    sets: int  # 0: one weight [N, K]; else [sets, N, K]
    N: int
    K: int
    fmt: int
    tensor_scale: Optional[torch.Tensor]


@functools.lru_cache(maxsize=None)
def _mx4_packed_bytes(sets: int, N: int, K: int, fmt: int) -> int:
    return int(load().egopq_mx4_packed_bytes(sets or 1, N, K, fmt))


def _mx4_packed(weight: Mx4Weight) -> int:
    """The records' address, of a weight that may have been put together by hand."""
    packed, sets, N, K, fmt, _ = weight
    need = _mx4_packed_bytes(sets, N, K, fmt)
    if packed.nbytes < need:
        raise ValueError(f"packed of {packed.nbytes} bytes, {need} needed")
    return _mx4_at(packed)


def mx4_quant(x: torch.Tensor, fmt: int = MX4_E8M0, tensor_scale: Optional[torch.Tensor] = None,
              gated: bool = False, with_codes: bool = True, with_tc: bool = True,
              out: Optional[Mx4Rows] = None, stream=None) -> Mx4Rows:
    """x [M, K] (bf16, fp16 or fp32) to 4-bit codes and block scales; gated: x is
    [M, 2K], and silu(x[:, :K]) * x[:, K:] is quantized (include/egopq.h has the
    formulas). tensor_scale fp32 [1]: MX4_E4M3 only. with_codes writes codes and
    scales, with_tc the form that mx4_gemm reads. `out`: rows of an earlier call of
    the same sizes."""
    block, kind = mx4_block(fmt), _mx4_type(x.dtype)
    M, K = x.shape
    if gated:
        if K % 2:
            raise ValueError(f"{K} gate and up values: an odd number")
        K //= 2
    lib = load()
    if out is None:
        dev = x.device
        codes = scales = a_tc = None
        if K % 32:
            raise EgopqError(-2, f"K ({K}) must be a multiple of 32")
        if with_codes:
            codes = _output((M, K // 2), torch.uint8, dev, stream)
            scales = _output((M, K // block), torch.uint8, dev, stream)
        if with_tc:
            a_tc = _output((int(lib.egopq_mx4_operand_bytes(M, K, fmt)),), torch.uint8, dev,
                           stream)
        out = Mx4Rows(codes, scales, a_tc, M, K, fmt, tensor_scale)
    else:
        if (out.M, out.K, out.fmt) != (M, K, fmt):
            raise ValueError(f"out holds {out.M} x {out.K} of format {out.fmt}, expected "
                             f"{M} x {K} of {fmt}")
        _mx4_rows_check(out)
        codes, scales, a_tc = out.codes, out.scales, out.a_tc
        _mx4_here(x, codes, scales, a_tc)
        out = out._replace(tensor_scale=tensor_scale)
    _mx4_here(x, tensor_scale)  # (what the call made itself needs no look)
    _check(lib.egopq_mx4_quant(
        _mx4_at(x), kind, M, K, fmt, None if tensor_scale is None else _mx4_scale(tensor_scale, 1),
        gated, None if codes is None else codes.data_ptr(),
        None if scales is None else scales.data_ptr(),
        None if a_tc is None else a_tc.data_ptr(), _stream(stream)))
    return out


def _mx4_rows_check(rows: Mx4Rows):
    """The sizes that a call relies on, of rows that may have been put together by
    hand."""
    M, K, block = rows.M, rows.K, mx4_block(rows.fmt)
    if rows.codes is not None:
        _arg(rows.codes, torch.uint8, M, K // 2)
    if rows.scales is not None:
        _arg(rows.scales, torch.uint8, M, K // block)
    if rows.a_tc is not None:
        need = int(load().egopq_mx4_operand_bytes(M, K, rows.fmt))
        _ptr(rows.a_tc)
        if rows.a_tc.nbytes < need:
            raise ValueError(f"a_tc of {rows.a_tc.nbytes} bytes, {need} needed")


def mx4_dequant(rows: Mx4Rows, dtype: Optional[torch.dtype] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values [M, K] that rows' codes and scales stand for: bf16 unless dtype or
    out says otherwise."""
    codes, scales, _, M, K, fmt, tensor_scale = rows
    if codes is None or scales is None:
        raise ValueError("rows without codes and scales (with_codes=False)")
    dtype = _mx4_result(dtype, out, torch.bfloat16)
    _mx4_here(codes, scales, tensor_scale, out)
    c = _arg(codes, torch.uint8, M, K // 2)
    s = _arg(scales, torch.uint8, M, K // mx4_block(fmt))
    if out is None:
        out = _output((M, K), dtype, codes.device, stream)
    _check(load().egopq_mx4_dequant(
        c, s, M, K, fmt, None if tensor_scale is None else _mx4_scale(tensor_scale, 1),
        _mx4_type(dtype), _arg(out, dtype, M, K), _stream(stream)))
    return out


def mx4_pack(codes: torch.Tensor, scales: torch.Tensor, fmt: int = MX4_E8M0,
             tensor_scale: Optional[torch.Tensor] = None, stream=None) -> Mx4Weight:
    """Pack 4-bit weights for the products: codes uint8 [N, K/2] and scales uint8
    [N, K/block] of one linear (as mx4_quant writes them), or [E, N, ..] of a
    layer's experts; tensor_scale fp32 [1] or [E] (MX4_E4M3 only)."""
    block = mx4_block(fmt)
    sets = codes.shape[0] if codes.dim() == 3 else 0
    N, K = codes.shape[-2], codes.shape[-1] * 2
    lead = (sets,) if sets else ()
    nbytes = int(load().egopq_mx4_packed_bytes(max(sets, 1), N, K, fmt))
    if codes.dim() not in (2, 3) or nbytes == 0:
        raise EgopqError(-2, f"codes of shape {tuple(codes.shape)} are not packable")
    if fmt == MX4_E8M0 and tensor_scale is not None:
        raise EgopqError(-1, "E8M0 blocks have no tensor scale")
    if tensor_scale is not None:
        _mx4_scale(tensor_scale, max(sets, 1))
    _mx4_here(codes, scales, tensor_scale)
    c = _arg(codes, torch.uint8, *lead, N, K // 2)
    s = _arg(scales, torch.uint8, *lead, N, K // block)
    packed = _output((nbytes,), torch.uint8, codes.device, stream)
    _check(load().egopq_mx4_pack(c, s, max(sets, 1), N, K, fmt, packed.data_ptr(),
                                 _stream(stream)))
    return Mx4Weight(packed, sets, N, K, fmt, tensor_scale)


def mx4_unpack(weight: Mx4Weight, stream=None) -> tuple:
    """(codes, scales) of a packed weight, as mx4_pack took them."""
    packed, sets, N, K, fmt, _ = weight
    _mx4_here(packed)
    at = _mx4_packed(weight)
    lead, dev = ((sets,) if sets else ()), packed.device
    codes = _output((*lead, N, K // 2), torch.uint8, dev, stream)
    scales = _output((*lead, N, K // mx4_block(fmt)), torch.uint8, dev, stream)
    _check(load().egopq_mx4_unpack(at, max(sets, 1), N, K, fmt, _ptr(codes),
                                   _ptr(scales), _stream(stream)))
    return codes, scales


def mx4_gemm(rows: Mx4Rows, weight: Mx4Weight, dtype: Optional[torch.dtype] = None,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows in 4 bits times a packed 4-bit weight: y [M, N], bf16 unless dtype or out
    says otherwise."""
    packed, sets, N, K, fmt, w_scale = weight
    if sets:
        raise ValueError("weights of several sets: mx4_linear_ragged")
    if (rows.K, rows.fmt) != (K, fmt):
        raise ValueError(f"rows of K={rows.K} format {rows.fmt}, a weight of K={K} format {fmt}")
    if rows.a_tc is None:
        raise ValueError("rows without the products' form (with_tc=False)")
    dtype = _mx4_result(dtype, out, torch.bfloat16)
    _mx4_here(packed, rows.a_tc, rows.tensor_scale, w_scale, out)
    _mx4_rows_check(rows)
    at = _mx4_packed(weight)
    if out is None:
        out = _output((rows.M, N), dtype, packed.device, stream)
    _check(load().egopq_mx4_gemm(_ptr(rows.a_tc), at, _mx4_scale(rows.tensor_scale, 1),
                                 _mx4_scale(w_scale, 1), rows.M, N, K, fmt, _mx4_type(dtype),
                                 _arg(out, dtype, rows.M, N), _stream(stream)))
    return out


def mx4_workspace(rows: int, weight: Mx4Weight, device, stream=None) -> torch.Tensor:
    """A workspace for mx4_linear or (a weight of several sets) mx4_linear_ragged
    of `rows` rows and of any fewer, of the stream it is to be used on."""
    n = int(load().egopq_mx4_linear_workspace_bytes(rows, weight.sets, weight.K, weight.fmt))
    return _scratch(n, torch.uint8, device, stream)


def _mx4_input(x: torch.Tensor, K: int, gated: bool) -> tuple:
    """Rows and type of a linear's input."""
    shape = x.shape
    if len(shape) != 2 or shape[1] != (2 * K if gated else K):
        raise ValueError(f"x of shape {tuple(shape)} for {'gated ' if gated else ''}K = {K}")
    return shape[0], _mx4_type(x.dtype)


def mx4_linear(x: torch.Tensor, weight: Mx4Weight, tensor_scale: Optional[torch.Tensor] = None,
               gated: bool = False, dtype: Optional[torch.dtype] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """mx4_quant of x [M, K] (gated: [M, 2K], gate and up halves) and the product
    with a packed 4-bit weight, in one call: y [M, N], of x's type unless dtype or
    out says otherwise. tensor_scale: the rows' (MX4_E4M3)."""
    packed, sets, N, K, fmt, w_scale = weight
    if sets:
        raise ValueError("weights of several sets: mx4_linear_ragged")
    M, x_type = _mx4_input(x, K, gated)
    dtype = _mx4_result(dtype, out, x.dtype)
    if out is None:
        out = _output((M, N), dtype, x.device, stream)
    if workspace is None:
        workspace = mx4_workspace(M, weight, x.device, stream)
    device = _mx4_here(x, packed, out, workspace, tensor_scale, w_scale)
    at = _mx4_packed(weight)
    _check(load().egopq_mx4_linear(
        _mx4_at(x), x_type, M, N, K, gated,
        None if tensor_scale is None else _mx4_scale(tensor_scale, 1), at,
        None if w_scale is None else _mx4_scale(w_scale, 1), fmt, _mx4_type(dtype),
        _arg(out, dtype, M, N), _mx4_at(workspace), workspace.nbytes,
        _mx4_stream(stream, device)))
    return out


def mx4_linear_ragged(x: torch.Tensor, offsets: torch.Tensor, weight: Mx4Weight,
                      index: Optional[torch.Tensor] = None,
                      tensor_scale: Optional[torch.Tensor] = None, gated: bool = False,
                      dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """mx4_linear of rows sorted by the weight they take: rows
    [offsets[e], offsets[e + 1]) (int32 [E + 1], on the device) times weight e of a
    weight of E sets. Row r is x's row r, or index[r] (int32 [rows]) of an x of any
    number of rows. y's other rows stay as they are: those of a y that the call
    makes are not written."""
    packed, sets, N, K, fmt, w_scale = weight
    if not sets:
        raise ValueError("a weight of several sets is needed (codes [E, N, K/2])")
    x_rows, x_type = _mx4_input(x, K, gated)
    rows = x_rows if index is None else index.shape[0]
    dtype = _mx4_result(dtype, out, x.dtype)
    if out is None:
        out = _output((rows, N), dtype, x.device, stream)
    if workspace is None:
        workspace = mx4_workspace(rows, weight, x.device, stream)
    device = _mx4_here(x, packed, out, workspace, offsets, index, tensor_scale, w_scale)
    at = _mx4_packed(weight)
    _check(load().egopq_mx4_linear_ragged(
        _mx4_at(x), x_type, x_rows, None if index is None else _arg(index, torch.int32, rows),
        _arg(offsets, torch.int32, sets + 1), rows, sets, N, K, gated,
        None if tensor_scale is None else _mx4_scale(tensor_scale, 1), at,
        None if w_scale is None else _mx4_scale(w_scale, sets), fmt, _mx4_type(dtype),
        _arg(out, dtype, rows, N), _mx4_at(workspace), workspace.nbytes,
        _mx4_stream(stream, device)))
    return out


def supported(M: int, N: int, K: int, variant: int = VARIANT_W4A8, group: int = GROUP) -> bool:
    return bool(load().egopq_supported(M, N, K, group, variant))


def device_status(stream=None) -> int:
    """Synchronize and return (and clear) the device error status code."""
    return int(load().egopq_device_status(_stream(stream)))


def selftest_timeout(timeout_us: int, stream=None) -> None:
    _check(load().egopq_selftest_timeout(timeout_us, _stream(stream)))


def version() -> int:
    return int(load().egopq_version())
