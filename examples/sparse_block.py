"""One block of a served sparse model: a projection with the adapters of many
requests beside it, then a mixture of experts, on packed int4 weights.

    python examples/sparse_block.py [--tokens 512] [--requests 33] [--variant w4a8|w4a16]

Every token belongs to a request and every request names an adapter (or none).
The block is
    h = x + W_o x + adapter(x)          one call: W4A8 projection and adapters
    l = R norm(h)                       router logits (plain bf16 matmul)
    out = h + sum_j w_j expert_j(norm(h))   moe_route, moe_experts
First it runs a batch of prompt tokens, then single tokens of all requests as
one CUDA graph, the way a server decodes; a few rows of both are checked against
the formulas in 64 bits. Weights are random; sizes come from the arguments.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import w4a8_quantized_gemm_gb300 as eg  # noqa: E402

G = eg.GROUP


def random_w4(rows, K, gen, device):
    """Random codes, scales and zero points of a [rows, K] int4 weight."""
    q = torch.randint(0, 16, (rows, K), generator=gen, device=device, dtype=torch.uint8)
    s = (torch.rand(rows, K // G, generator=gen, device=device) + 0.5) / (4.6 * K ** 0.5)
    z = torch.randint(7, 10, (rows, K // G), generator=gen, device=device, dtype=torch.uint8)
    return q, s.half(), z


class SparseBlock:
    """Packed weights, adapters and the buffers for up to `max_tokens` tokens."""

    def __init__(self, hidden, inner, experts, picks, adapters, rank, max_tokens, variant, seed,
                 device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.H, self.I, self.E, self.k = hidden, inner, experts, picks
        self.variant = variant
        H, I, E, L = hidden, inner, experts, adapters
        self.o_w4 = random_w4(H, H, g, device)
        self.o = eg.pack_w4(*self.o_w4)
        gu, dn = random_w4(E * 2 * I, H, g, device), random_w4(E * H, I, g, device)
        self.gate_up_w4 = [t.view(E, 2 * I, -1) for t in gu]
        self.down_w4 = [t.view(E, H, -1) for t in dn]
        self.layer = eg.moe_pack(*self.gate_up_w4, *self.down_w4)
        self.router = (2 * torch.randn(E, H, generator=g, device=device) / H ** 0.5).bfloat16()
        A = (torch.randn(L, rank, H, generator=g, device=device) / H ** 0.5).bfloat16()
        B = (torch.randn(L, H, rank, generator=g, device=device) / rank ** 0.5).bfloat16()
        ranks = torch.randint(1, rank + 1, (L,), generator=g, device=device, dtype=torch.int32)
        self.adapters = eg.LoraAdapters(A, B, torch.full((L,), 0.5, device=device), ranks)
        # workspaces of the largest batch; any fewer tokens fit
        self.ws_o = eg.w4a8_linear_lora_workspace(max_tokens, H, H, self.adapters, device)
        self.ws_moe = eg.moe_workspace(max_tokens, picks, E, H, I, variant, device)

    def norm(self, h):
        return torch.nn.functional.rms_norm(h, (self.H,))

    def forward(self, x, adapter_of_token):
        """x bf16 [T, H], adapter_of_token int32 [T] (-1: none) -> (out, h, ids, weights)."""
        h = x + eg.w4a8_linear_lora(x, self.o, self.H, self.adapters, adapter_of_token,
                                    workspace=self.ws_o)
        n = self.norm(h)
        weights, ids = eg.moe_route(n @ self.router.t(), self.k)
        out = h + eg.moe_experts(n, ids, weights, self.layer, variant=self.variant,
                                 workspace=self.ws_moe)
        return out, h, ids, weights


def dequant(w4, rows=slice(None)):
    q, s, z = (t[rows].double() for t in w4)
    return (q - z.repeat_interleave(G, -1)) * s.repeat_interleave(G, -1)


def codes(x, variant):
    """What the products see of x: itself, or its int8 codes times their scale."""
    if variant == eg.VARIANT_W4A16:
        return x.double()
    s = x.float().abs().amax(-1, keepdim=True) / 127
    return torch.where(s > 0, torch.round(x.float() / s), 0).double() * s.double()


def check(block, x, adapter_of_token, result, rows):
    """Relative 2-norm distance of a few rows from the formulas in 64 bits."""
    out, h, ids, weights = result
    ad = block.adapters
    o = dequant(block.o_w4)
    worst = 0.0
    for t in rows:
        y = codes(x[t], eg.VARIANT_W4A8) @ o.t()
        a = int(adapter_of_token[t])
        if a >= 0:
            r = int(ad.ranks[a])
            y = y + float(ad.scale[a]) * (ad.B[a, :, :r].double()
                                          @ (ad.A[a, :r].double() @ x[t].double()))
        ref_h = x[t].double() + y
        worst = max(worst, ((h[t] - ref_h).norm() / ref_h.norm()).item())
        n = block.norm(h[t:t + 1])[0]
        scores = torch.softmax((block.norm(h) @ block.router.t())[t].double(), -1)
        best = scores.topk(block.k)
        assert torch.allclose(best.values / best.values.sum(), weights[t].double(), rtol=1e-5)
        m = torch.zeros(block.H, dtype=torch.float64, device=x.device)
        for w, e in zip(weights[t].double(), ids[t].tolist()):
            gu = codes(n, block.variant) @ dequant(block.gate_up_w4, e).t()
            v = torch.nn.functional.silu(gu[:block.I]) * gu[block.I:]
            m += w * (codes(v.bfloat16(), block.variant) @ dequant(block.down_w4, e).t())
        ref = h[t].double() + m
        worst = max(worst, ((out[t] - ref).norm() / ref.norm()).item())
    return worst


def timed(fn, n=20):
    for _ in range(3):
        fn()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    t0.record()
    for _ in range(n):
        fn()
    t1.record()
    torch.cuda.synchronize()
    return t0.elapsed_time(t1) / n * 1e3


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--tokens", type=int, default=512, help="prompt tokens of the batch")
    p.add_argument("--requests", type=int, default=33, help="requests, one token each when decoding")
    p.add_argument("--hidden", type=int, default=3584)
    p.add_argument("--inner", type=int, default=1280)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--picks", type=int, default=8)
    p.add_argument("--adapters", type=int, default=16)
    p.add_argument("--rank", type=int, default=32)
    p.add_argument("--variant", choices=["w4a8", "w4a16"], default="w4a8")
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    variant = eg.VARIANT_W4A8 if a.variant == "w4a8" else eg.VARIANT_W4A16
    block = SparseBlock(a.hidden, a.inner, a.experts, a.picks, a.adapters, a.rank,
                        max(a.tokens, a.requests), variant, a.seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(a.seed + 1)
    # every third request has no adapter
    adapter = torch.randint(0, a.adapters, (a.requests,), generator=g, device="cuda",
                            dtype=torch.int32)
    adapter[::3] = -1
    of_token = adapter[torch.arange(a.tokens, device="cuda") * a.requests // max(a.tokens, 1)]

    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    prompt = block.forward(x, of_token)
    errors = [check(block, x, of_token, prompt, {0, a.tokens // 2, a.tokens - 1})]
    us = timed(lambda: block.forward(x, of_token))
    print(f"prompt: {a.tokens} tokens of {a.requests} requests, {us:.1f} us, "
          f"error {errors[-1]:.4f}")

    x1 = torch.randn(a.requests, a.hidden, generator=g, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(x1, adapter)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = block.forward(x1, adapter)
    x1.copy_(torch.randn(a.requests, a.hidden, generator=g, device="cuda"))
    graph.replay()
    errors.append(check(block, x1, adapter, step, {0, a.requests // 2, a.requests - 1}))
    us = timed(graph.replay)
    print(f"decode: {a.requests} requests a step, one graph, {us:.1f} us, error {errors[-1]:.4f}")
    if eg.device_status() != 0:
        raise RuntimeError("a kernel reported an error")
    return errors


if __name__ == "__main__":
    # three roundings to bf16 a result, each about 0.42 * 2^-8 of it, and codes
    # that the fp32 sums move by one: well inside 1 %
    sys.exit(0 if max(main()) < 1e-2 else 1)
