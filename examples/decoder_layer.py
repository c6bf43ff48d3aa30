"""A decoder layer with routed experts, run a prompt in chunks and then token by
token: residual norm -> NVFP4 projection of queries, keys and values -> rotation
and append to the paged 8-bit cache -> attention -> NVFP4 output projection ->
residual norm -> router -> routed experts.

Every step is one of the library's kernels; a decode step is captured once as a
CUDA graph and replayed (its sequence lengths are device arrays that the graph
itself advances).  Weights are random.

    python examples/decoder_layer.py --batch 8 --prompt 300 --tokens 32
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from quantized_moe_routed_gb300 import KVCache, MoePlan, Nvfp4Linear, add_rms_norm, rope_table  # noqa: E402
from quantized_moe_routed_gb300.inputs import Workload, make_expert_weights, quantize_nvfp4  # noqa: E402
from quantized_moe_routed_gb300.layer import PAGE  # noqa: E402


class DecoderLayer:
    """H: hidden size; I, E, k: the experts' inner size, their number, experts a token."""

    def __init__(self, H=512, I=256, E=8, k=4, q_heads=8, kv_heads=2, head_dim=64, n_pages=64, positions=4096,
                 T_max=512, device="cuda:0", seed=0):
        gen = torch.Generator().manual_seed(seed)

        def linear(n, m, gain):
            w = torch.randn((n, m), generator=gen) * (gain / m ** 0.5)
            q, s, ts = quantize_nvfp4(w)
            return Nvfp4Linear(q.to(device), s.to(device), ts.reshape(1).float().to(device))

        self.H, self.heads, self.device = H, (q_heads, kv_heads, head_dim), torch.device(device)
        self.norm1 = torch.rand(H, generator=gen).add_(0.5).bfloat16().to(device)
        self.norm2 = torch.rand(H, generator=gen).add_(0.5).bfloat16().to(device)
        self.qkv = linear((q_heads + 2 * kv_heads) * head_dim, H, 1.0)
        self.out = linear(H, q_heads * head_dim, 1.0)
        self.router = linear(E, H, 1.0)
        self.cache = KVCache(n_pages, q_heads, kv_heads, head_dim, rope=rope_table(positions, head_dim, device=device),
                             device=device)
        wl = Workload("layer", T=1, H=H, I=I, E=E, k=k, routing="uniform", seed=seed)
        weights = {name: t.to(device) for name, t in make_expert_weights(wl).items()}
        self.experts = MoePlan(weights, H, I, E, k, T_max=T_max, strict=True)
        self.cache_ws, self.experts_ws = self.cache.new_workspace(), self.experts.new_workspace()

    def __call__(self, x, residual, q_off, kv_len, pages, max_q):
        """x: the layer before's output, float32 or bfloat16 [N, H]; residual:
        bfloat16 [N, H], updated in place.  Returns this layer's output, float32."""
        hq, hkv, d = self.heads
        h = add_rms_norm(x, self.norm1, residual=residual)
        q, k, v = self.qkv(h, dtype=torch.bfloat16).view(-1, hq + 2 * hkv, d).split((hq, hkv, hkv), dim=1)
        step = (q_off, kv_len, pages, self.cache_ws, max_q)
        q = self.cache.append(k, v, *step, q=q)
        o = self.cache.attend(q, *step)
        h = add_rms_norm(self.out(o.view(-1, hq * d)), self.norm2, residual=residual)
        return self.experts.step_logits(h, self.router(h), self.experts_ws)

    def check(self):
        """0, or the first device status of the cache's and the experts' work."""
        return self.cache.check(self.cache_ws) or self.experts.check(self.experts_ws)


class Session:
    """B sequences over a layer's cache, with room for max_len tokens each."""

    def __init__(self, layer: DecoderLayer, B: int, max_len: int):
        self.layer, self.B, dev = layer, B, layer.device
        per = (max_len + PAGE - 1) // PAGE
        if B * per > layer.cache.n_pages:
            raise ValueError(f"{B} sequences of {max_len} tokens need {B * per} pages, the cache has {layer.cache.n_pages}")
        self.pages = torch.randperm(layer.cache.n_pages, device=dev)[:B * per].int().view(B, per).contiguous()
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.one = torch.arange(B + 1, dtype=torch.int32, device=dev)

    def prefill(self, x, chunk=128):
        """x bfloat16 [B, n, H] -> the layer's output at the last position, [B, H]."""
        n = x.shape[1]
        for at in range(0, n, chunk):
            m = min(chunk, n - at)
            part = x[:, at:at + m].reshape(self.B * m, -1)
            self.kv_len += m
            y = self.layer(part, torch.zeros_like(part), self.one * m, self.kv_len, self.pages, m)
        return y.view(self.B, m, -1)[:, -1]

    def capture(self):
        """A graph of one decode step: reads self.x, writes self.y."""
        self.x = torch.zeros((self.B, self.layer.H), dtype=torch.bfloat16, device=self.layer.device)
        self.residual = torch.zeros_like(self.x)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = self.decode(self.x, self.residual)

    def decode(self, x, residual):
        residual.zero_()
        self.kv_len += 1
        return self.layer(x, residual, self.one, self.kv_len, self.pages, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--tokens", type=int, default=32)
    args = ap.parse_args()
    max_len = args.prompt + args.tokens
    layer = DecoderLayer(n_pages=args.batch * (max_len // PAGE + 1), positions=max_len, T_max=args.batch * 128)
    s = Session(layer, args.batch, max_len)
    y = s.prefill(torch.randn((args.batch, args.prompt, layer.H), device=layer.device).bfloat16())
    s.capture()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(args.tokens):
        s.x.copy_(y)
        s.graph.replay()
        y = s.y
    end.record()
    status = layer.check()
    print(f"status {status}, {args.batch} sequences of {int(s.kv_len[0])} tokens, "
          f"{start.elapsed_time(end) / max(args.tokens, 1) * 1e3:.1f} us a decode step, |y| {float(y.abs().mean()):.4f}")
    return status


if __name__ == "__main__":
    sys.exit(main())
