"""The binding's own part of a call, without a device: a library that only notes
its arguments, CPU tensors in the place of device ones, and the allocator's
streams noted as torch is asked for them."""
import contextlib

import pytest
import torch

import w4a8_quantized_gemm_gb300 as eg

BF16, U8, I32, F32, F16 = (torch.bfloat16, torch.uint8, torch.int32, torch.float32,
                           torch.float16)


class Library:
    """Answers every entry point: sizes with 4096 bytes, calls with success."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_bytes") else 0
        return call

    def args(self, name):
        return [a for n, a in self.calls if n == name][-1]


class Streams:
    """What torch.cuda would be asked: the stream an allocation is made on, and
    the streams each tensor is recorded on besides."""

    def __init__(self):
        self.current, self.made, self.recorded = "caller", [], {}

    @contextlib.contextmanager
    def on(self, stream):
        was, self.current = self.current, stream
        yield
        self.current = was


class Side:
    cuda_stream = 0x5150


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(eg, "load", lambda: lib)
    monkeypatch.setattr(eg, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(eg, "_stream", lambda s=None: 0 if s is None else s.cuda_stream)
    return lib


@pytest.fixture
def streams(monkeypatch):
    st = Streams()
    empty, empty_like = torch.empty, torch.empty_like

    def noted(make):
        def call(*a, **kw):
            t = make(*a, **kw)
            st.made.append((t, st.current))
            return t
        return call

    monkeypatch.setattr(torch, "empty", noted(empty))
    monkeypatch.setattr(torch, "empty_like", noted(empty_like))
    monkeypatch.setattr(torch.cuda, "stream", st.on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: st.current)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: st.recorded.setdefault(id(t), []).append(s))
    return st


def zeros(*shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def adapters(L=2, r=8, K=128, N=128):
    return eg.LoraAdapters(zeros(L, r, K, dtype=BF16), zeros(L, N, r, dtype=BF16),
                           zeros(L, dtype=F32), zeros(L, dtype=I32))


def calls():
    """name -> a call of it with `stream`, returning the tensors it hands out."""
    M, N, K = 3, 128, 128
    x = zeros(M, K, dtype=BF16)
    packed = zeros(4096, dtype=U8)
    w4 = (zeros(N, K, dtype=U8), zeros(N, 1, dtype=F16), zeros(N, 1, dtype=U8))
    act = eg.QuantAct(zeros(M, K, dtype=torch.int8), zeros(M, dtype=F32), zeros(M, 1, dtype=I32),
                      zeros(4096, dtype=U8))
    w8, s8 = zeros(N, K, dtype=torch.int8), zeros(N, dtype=F16)
    ids, wt = zeros(M, 2, dtype=I32), zeros(M, 2, dtype=F32)
    layer = eg.MoeLayer(packed, packed, 4, 128, 128)
    experts = (zeros(2, 256, 128, dtype=U8), zeros(2, 256, 1, dtype=F16),
               zeros(2, 256, 1, dtype=U8), zeros(2, 128, 128, dtype=U8),
               zeros(2, 128, 1, dtype=F16), zeros(2, 128, 1, dtype=U8))
    one = lambda t: [t]
    return {
        "pack_w4": lambda s: one(eg.pack_w4(*w4, stream=s)),
        "unpack_w4": lambda s: list(eg.unpack_w4(packed, N, K, stream=s)),
        "pack_w4_gptq": lambda s: one(eg.pack_w4_gptq(
            zeros(K // 8, N, dtype=I32), zeros(1, N // 8, dtype=I32), zeros(1, N, dtype=F16),
            stream=s)),
        "dequant_w4": lambda s: one(eg.dequant_w4(packed, N, K, stream=s)),
        "quant_act": lambda s: list(eg.quant_act(x, stream=s)),
        "w4a8_gemm": lambda s: one(eg.w4a8_gemm(act, packed, N, K, stream=s)),
        "w4a8_linear": lambda s: one(eg.w4a8_linear(x, packed, N, stream=s)),
        "w4a8_gemm_grouped": lambda s: eg.w4a8_gemm_grouped(act, [packed] * 2, [N] * 2, K,
                                                            stream=s),
        "w4a8_linear_grouped": lambda s: eg.w4a8_linear_grouped(x, [packed] * 2, [N] * 2,
                                                                stream=s),
        "w4a8_group_partials": lambda s: one(eg.w4a8_group_partials(act, packed, N, K, stream=s)),
        "w4a16_gemm": lambda s: one(eg.w4a16_gemm(x, packed, N, K, stream=s)),
        "w8a16_gemm": lambda s: one(eg.w8a16_gemm(x, w8, s8, stream=s)),
        "w8a8_gemm": lambda s: one(eg.w8a8_gemm(act, w8, s8, stream=s)),
        "bf16_gemm_twin": lambda s: one(eg.bf16_gemm_twin(x, zeros(N, K, dtype=BF16), stream=s)),
        "moe_route": lambda s: list(eg.moe_route(zeros(M, 4, dtype=F32), 2, stream=s)),
        "moe_pack": lambda s: list(eg.moe_pack(*experts, stream=s)[:2]),
        "moe_experts": lambda s: one(eg.moe_experts(x, ids, wt, layer, stream=s)),
        "lora_add": lambda s: one(eg.lora_add(zeros(M, N, dtype=BF16), x, adapters(),
                                              zeros(M, dtype=I32), stream=s)),
        "w4a8_linear_lora": lambda s: one(eg.w4a8_linear_lora(x, packed, N, adapters(),
                                                              zeros(M, dtype=I32), stream=s)),
    }


NAMES = ["pack_w4", "unpack_w4", "pack_w4_gptq", "dequant_w4", "quant_act", "w4a8_gemm",
         "w4a8_linear", "w4a8_gemm_grouped", "w4a8_linear_grouped", "w4a8_group_partials",
         "w4a16_gemm", "w8a16_gemm", "w8a8_gemm", "bf16_gemm_twin", "moe_route", "moe_pack",
         "moe_experts", "lora_add", "w4a8_linear_lora"]


def test_every_call_with_a_stream_is_listed(lib):
    assert sorted(calls()) == sorted(NAMES)


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream_is_of_that_stream(lib, streams, name):
    """A workspace is dropped as the call returns, with its kernels still
    queued: it has to come from the memory of the stream they run on. So do the
    outputs, which the caller's stream may then read."""
    side = Side()
    handed = calls()[name](side)
    assert streams.made and all(s is side for _, s in streams.made)
    assert lib.calls[-1][1][-1] == side.cuda_stream
    for t in handed:
        assert streams.recorded.get(id(t)) == ["caller"]
    # scratch memory is read by no other stream and waits for none
    kept = {id(t) for t in handed}
    assert all(id(t) in kept or id(t) not in streams.recorded for t, _ in streams.made)


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_the_current_stream(lib, streams, name):
    calls()[name](None)
    assert all(s == "caller" for _, s in streams.made) and not streams.recorded


def test_workspaces_can_be_made_for_another_stream(lib, streams):
    side = Side()
    eg.moe_workspace(3, 2, 4, 128, 128, eg.VARIANT_W4A8, "cpu", stream=side)
    eg.lora_workspace(3, 128, 128, adapters(), "cpu", stream=side)
    eg.w4a8_linear_lora_workspace(3, 128, 128, adapters(), "cpu", stream=side)
    assert [s for _, s in streams.made] == [side] * 3


# ------------------------------------------------- adapters whose memory is replaced ---

def lora_calls(ad):
    """(name, the four addresses it passes on) for each call that takes adapters."""
    M = 3
    x, y, ids = (zeros(M, ad.K, dtype=BF16), zeros(M, ad.N, dtype=BF16), zeros(M, dtype=I32))
    return [("egopq_lora_add", slice(2, 6), lambda: eg.lora_add(y, x, ad, ids)),
            ("egopq_w4a8_linear_lora", slice(2, 6),
             lambda: eg.w4a8_linear_lora(x, zeros(4096, dtype=U8), ad.N, ad, ids))]


@pytest.mark.parametrize("which", ["A", "B", "scale", "ranks"])
@pytest.mark.parametrize("call", [0, 1])
def test_adapters_follow_memory_that_was_replaced(lib, which, call):
    ad = adapters()
    name, at, run = lora_calls(ad)[call]
    run()
    tensors = [ad.A, ad.B, ad.scale, ad.ranks]
    assert list(lib.args(name)[at]) == [t.data_ptr() for t in tensors]
    t = getattr(ad, which)
    before = t.data_ptr()
    t.data = t.data.clone()
    assert t.data_ptr() != before
    run()
    assert list(lib.args(name)[at]) == [t.data_ptr() for t in tensors]


@pytest.mark.parametrize("which", ["A", "B", "scale", "ranks"])
@pytest.mark.parametrize("call", [0, 1])
def test_adapters_whose_memory_no_longer_fits_are_refused(lib, which, call):
    for broken in (lambda t: t[:1].clone(), lambda t: t.double().to(torch.int16)):
        ad = adapters()
        name, _, run = lora_calls(ad)[call]
        t = getattr(ad, which)
        t.data = broken(t)
        with pytest.raises((ValueError, TypeError)):
            run()
        assert name not in [n for n, _ in lib.calls]


def test_adapters_keep_the_memory_they_were_checked_with(lib):
    """Else new memory at the address of the old could pass for it."""
    ad = adapters()
    assert {s.data_ptr() for s in ad._kept} == {t.data_ptr() for t in
                                                (ad.A, ad.B, ad.scale, ad.ranks)}
    old = ad.A.data_ptr()
    ad.A.data = ad.A.data.clone()
    assert old in {s.data_ptr() for s in ad._kept}
    lora_calls(ad)[0][2]()
    assert old not in {s.data_ptr() for s in ad._kept}
