"""A layer of routed experts with float8 or 4-bit weights, from one decoded token to a prefill batch.

  python examples/moe_layer.py [--experts 64] [--top-k 8] [--hidden 4096] [--inter 2048] [--tokens 1,16,256,4096]
                               [--format fp8 | fp4-16 | fp4-32]

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


class Float8:
    """e4m3 codes, a scale for each block of 128."""
    name, bits, off = "e4m3", 8, 2.0 ** -4       # half a step of a code, relative

    def weights(self, w):
        return q8.q8_quantize_weight_fp8(w)

    def tokens(self, x, slots):
        return q8.q8_quantize_fp8(x, slots=slots)

    def gated(self, h):
        return q8.q8_swiglu_quantize_fp8(h)

    def product(self, tokens, weights, offsets, dtype):
        return q8.q8_gemm_fp8_grouped(*tokens, *weights, offsets, out_dtype=dtype)

    def values(self, weights, e):
        """One expert's weights in 64 bits."""
        q, s = weights
        full = s[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return q[e].double() * full[:q.shape[1], :q.shape[2]]


class Float4:
    """e2m1 codes, a scale for each block of 16 or 32."""
    name, off = "e2m1", 2.0 ** -2                # half a step between 1 and 2, the coarsest relative one

    def __init__(self, block):
        self.block, self.bits = block, 4 + 8 / block

    def weights(self, w):
        return q8.q8_quantize_weight_fp4(w, block=self.block)

    def tokens(self, x, slots):
        return q8.q8_quantize_fp4(x, block=self.block, slots=slots)

    def gated(self, h):
        return q8.q8_swiglu_quantize_fp4(h, block=self.block)

    def product(self, tokens, weights, offsets, dtype):
        return q8.q8_gemm_fp4_grouped(*tokens, *weights, offsets, out_dtype=dtype)

    def values(self, weights, e):
        q, sf, s = weights
        return q8.q8_dequantize_fp4(q[e], sf[e], None if s is None else s[e], out_dtype=torch.float32).double()


FORMATS = {"fp8": Float8, "fp4-16": lambda: Float4(16), "fp4-32": lambda: Float4(32)}


class MoeLayer:
    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, bias: torch.Tensor, top_k: int, fmt=None):
        """w13 [E, 2 I, H] (gate rows, then up rows), w2 [E, H, I], bias fp32 [E]; fmt: one of FORMATS' (default float8)."""
        self.fmt = fmt or Float8()
        self.w13 = self.fmt.weights(w13)
        self.w2 = self.fmt.weights(w2)
        self.bias, self.top_k, self.experts = bias, top_k, w13.shape[0]

    def route(self, logits):
        return q8.q8_moe_route(logits, self.top_k, score="sigmoid", bias=self.bias, renorm=True)

    def __call__(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """x [T, H] bf16 or fp16, logits [T, E] -> [T, H]."""
        idx, weights = self.route(logits)
        offsets, slots = q8.q8_moe_plan(idx, self.experts)
        h = self.fmt.product(self.fmt.tokens(x, slots), self.w13, offsets, x.dtype)
        return q8.q8_moe_combine(self.fmt.product(self.fmt.gated(h), self.w2, offsets, x.dtype), slots, weights)

    def exact(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """The layer for a few tokens in 64 bits, without the quantization of the activations."""
        idx, weights = self.route(logits)
        y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        for t in range(x.shape[0]):
            for e, w in zip(idx[t].tolist(), weights[t].double()):
                if e >= 0:
                    gate, up = (self.fmt.values(self.w13, e) @ x[t].double()).chunk(2)
                    y[t] += w * (self.fmt.values(self.w2, e) @ (gate * torch.sigmoid(gate) * up))
        return y


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


def run(argv=None):
    """(the largest distance from 64 bits, what the format allows it to be)."""
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--top-k", type=int, default=8)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inter", type=int, default=2048)
    p.add_argument("--tokens", default="1,16,256,4096")
    p.add_argument("--format", choices=sorted(FORMATS), default="fp8")
    p.add_argument("--hbm-gbs", type=float, default=6781.8, help="copy bandwidth the weights' time is taken at")
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)
    E, H, I = a.experts, a.hidden, a.inter
    w13 = torch.randn((E, 2 * I, H), generator=g, device="cuda", dtype=torch.bfloat16) * H ** -0.5
    w2 = torch.randn((E, H, I), generator=g, device="cuda", dtype=torch.bfloat16) * I ** -0.5
    layer = MoeLayer(w13, w2, 0.1 * torch.randn(E, generator=g, device="cuda"), a.top_k, FORMATS[a.format]())
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
        floor = active * 3 * H * I * layer.fmt.bits / 8 / a.hbm_gbs / 1e3
        print(f"{T:6d} tokens: {us:9.1f} us a layer, {active} experts' weights {floor:7.1f} us, "
              f"off from 64 bits {off:.4f} (activations in {layer.fmt.name})")
    assert q8.q8_device_error() == 0
    return worst, layer.fmt.off


def main(argv=None):
    return run(argv)[0]


if __name__ == "__main__":
    # two roundings of activations (e4m3: 2^-4 at most, 2^-5.8 on average, each; e2m1: 2^-2 and 2^-3.4) and bf16 outputs
    worst, most = run()
    sys.exit(0 if worst < most else 1)
