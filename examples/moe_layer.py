"""A layer of routed experts with float8 weights, from one decoded token to a prefill batch.

  python examples/moe_layer.py [--experts 64] [--top-k 8] [--hidden 4096] [--inter 2048] [--tokens 1,16,256,4096]

Router (sigmoid scores, a balance bias), the experts' rows, tokens quantized into them, gate/up product,
gated activation with quantization, down product, weighted sum back: seven calls of the library, no
synchronisation between them, captured in a CUDA graph. For each batch size it prints the time of the
layer, the time that the active experts' weights take to be read at the measured copy bandwidth, and the distance
of some tokens' outputs from the same layer in 64 bits on the dequantized weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_quantized_gemm_gb300 as q8  # noqa: E402


class MoeLayer:
    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, bias: torch.Tensor, top_k: int):
        """w13 [E, 2 I, H] (gate rows, then up rows), w2 [E, H, I], bias fp32 [E]."""
        self.w13 = q8.q8_quantize_weight_fp8(w13)
        self.w2 = q8.q8_quantize_weight_fp8(w2)
        self.bias, self.top_k, self.experts = bias, top_k, w13.shape[0]

    def route(self, logits):
        return q8.q8_moe_route(logits, self.top_k, score="sigmoid", bias=self.bias, renorm=True)

    def __call__(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """x [T, H] bf16 or fp16, logits [T, E] -> [T, H]."""
        idx, weights = self.route(logits)
        offsets, slots = q8.q8_moe_plan(idx, self.experts)
        qa, sa = q8.q8_quantize_fp8(x, slots=slots)
        h = q8.q8_gemm_fp8_grouped(qa, sa, *self.w13, offsets, out_dtype=x.dtype)
        qh, sh = q8.q8_swiglu_quantize_fp8(h)
        return q8.q8_moe_combine(q8.q8_gemm_fp8_grouped(qh, sh, *self.w2, offsets, out_dtype=x.dtype), slots, weights)

    def exact(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """The layer for a few tokens in 64 bits, without the quantization of the activations."""
        idx, weights = self.route(logits)
        y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        for t in range(x.shape[0]):
            for e, w in zip(idx[t].tolist(), weights[t].double()):
                if e >= 0:
                    gate, up = (_values(*self.w13, e) @ x[t].double()).chunk(2)
                    y[t] += w * (_values(*self.w2, e) @ (gate * torch.sigmoid(gate) * up))
        return y


def _values(q, s, e):
    full = s[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return q[e].double() * full[:q.shape[1], :q.shape[2]]


def timed(layer, x, logits, replays=20):
    layer(x, logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, logits)
    for _ in range(3):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(replays):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return y, start.elapsed_time(end) * 1e3 / replays


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--top-k", type=int, default=8)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inter", type=int, default=2048)
    p.add_argument("--tokens", default="1,16,256,4096")
    p.add_argument("--hbm-gbs", type=float, default=6781.8, help="copy bandwidth the weights' time is taken at")
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)
    E, H, I = a.experts, a.hidden, a.inter
    w13 = torch.randn((E, 2 * I, H), generator=g, device="cuda", dtype=torch.bfloat16) * H ** -0.5
    w2 = torch.randn((E, H, I), generator=g, device="cuda", dtype=torch.bfloat16) * I ** -0.5
    layer = MoeLayer(w13, w2, 0.1 * torch.randn(E, generator=g, device="cuda"), a.top_k)
    del w13, w2
    worst = 0.0
    for T in (int(v) for v in a.tokens.split(",")):
        x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        logits = torch.randn((T, E), generator=g, device="cuda")
        y, us = timed(layer, x, logits)
        few = min(T, 4)
        want = layer.exact(x[:few], logits[:few])
        off = float((y[:few].double() - want).norm() / want.norm())
        worst = max(worst, off)
        active = int(torch.unique(layer.route(logits)[0]).numel())
        floor = active * 3 * H * I / a.hbm_gbs / 1e3
        print(f"{T:6d} tokens: {us:9.1f} us a layer, {active} experts' weights {floor:7.1f} us, "
              f"off from 64 bits {off:.4f} (activations in e4m3)")
    assert q8.q8_device_error() == 0
    return worst


if __name__ == "__main__":
    # two roundings of activations to e4m3 (2^-4 at most, 2^-5.8 on average, each) and bf16 outputs
    sys.exit(0 if main() < 2.0 ** -4 else 1)
