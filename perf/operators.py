"""Workloads of the float8 and routed-expert operators: what is measured, and their plain forms.

The cases are the steps of one layer of routed experts with float8 weights (routing, quantizing the
tokens into expert order, the experts' products, the gated activation, the weighted sum back) and the
float8 linear layer itself, from one token to prefill batches. `run` computes a step in elementary
torch operations (own = False) or through the package's entry points (own = True).
"""
import math

import torch

own = False

BLOCK = 128          # one scale for each block of 128 along K; 128 x 128 for weights
E4M3_MAX = 448.0
TINY = 1e-30         # the smallest block maximum a scale is made from
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def _cdiv(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through a router with grouped experts and a balance bias: launch latency
        dict(name="route 1 of 256", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             renorm=True, scale=2.5, dtype="fp32", masked=False),
        # a prefill batch through the same router
        dict(name="route 8192 of 256", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, renorm=True, scale=2.5, dtype="fp32", masked=False),
        # the activations of the int8 prefill16k layer, quantized to float8 instead
        dict(name="quantize 8192x16384", op="quantize", M=8192, K=16384, k=0, dtype="fp32"),
        # an odd batch of bf16 tokens written once into each of its experts' slots
        dict(name="quantize 1037x4096 to 8 slots", op="quantize", M=1037, K=4096, k=8, dtype="bf16"),
        # the gated activation between the experts' two products
        dict(name="swiglu 32768x2048", op="swiglu", M=32768, K=2048, dtype="bf16"),
        # the decode layer of the framework's own benchmark, with float8 weights
        dict(name="gemm 16x28672x8192", op="gemm", M=16, N=28672, K=8192, dtype="bf16"),
        # a ragged shape: no dimension is a multiple of a tile, the last scale blocks are short
        dict(name="gemm 517x2056x4112", op="gemm", M=517, N=2056, K=4112, dtype="fp32"),
        # the prefill layer of the framework's own benchmark
        dict(name="gemm 8192x8192x16384", op="gemm", M=8192, N=8192, K=16384, dtype="bf16"),
        # a decode batch of 16 tokens to 8 of 64 experts: every active expert's weights are read for a few rows
        dict(name="experts 128 rows of 64", op="grouped", rows=128, E=64, N=4096, K=4096, skew=0.5, dtype="bf16"),
        # a prefill batch of 4096 tokens to 8 of 64 experts, unevenly spread
        dict(name="experts 32768 rows of 64", op="grouped", rows=32768, E=64, N=4096, K=4096, skew=0.5, dtype="bf16"),
        # the experts' answers of a small batch summed back
        dict(name="combine 16x4096", op="combine", T=16, N=4096, k=8, dtype="bf16"),
        # and of a prefill batch
        dict(name="combine 8192x4096", op="combine", T=8192, N=4096, k=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "quantize", "quantize", "swiglu", "gemm", "gemm", "gemm", "grouped", "grouped",
                     "grouped", "combine"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * max(2, _log(rng, 8, 512) // n_group)
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(16, E // n_group * topk_group))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, n_group=n_group, topk_group=topk_group, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), masked=rng.random() < 0.4)
    if op == "quantize":
        k = rng.choice([0, 0, 1, 4, 8])
        K = 16 * _log(rng, 4, 1024)
        return dict(op=op, M=_log(rng, 1, min(32768, (1 << 27) // (K * max(1, k)))), K=K, k=k, dtype=dtype)
    if op == "swiglu":
        K = 16 * _log(rng, 4, 512)
        return dict(op=op, M=_log(rng, 1, min(65536, (1 << 26) // K)), K=K, dtype=dtype)
    if op == "gemm":
        K = 16 * _log(rng, 8, 1024)
        N = _log(rng, 64, min(28672, (1 << 28) // K))
        M = _log(rng, 1, min(8192, (1 << 39) // (N * K)))
        return dict(op=op, M=M, N=N, K=K, dtype=dtype)
    if op == "grouped":
        E = _log(rng, 2, 128)
        K = 16 * _log(rng, 16, 256)
        N = _log(rng, 64, min(8192, (1 << 30) // (E * K)))
        rows = _log(rng, 1, min(32768, (1 << 38) // (N * K)))
        return dict(op=op, rows=rows, E=E, N=N, K=K, skew=rng.choice([0.0, 0.5, 1.0]), dtype=dtype)
    N = 8 * _log(rng, 8, 1024)
    k = rng.choice([1, 2, 4, 6, 8])
    return dict(op=op, T=_log(rng, 1, min(16384, (1 << 28) // (N * k))), N=N, k=k, dtype=dtype)


def _counts(c):
    """Rows of each expert before the experts are shuffled: shares falling as a power of the rank."""
    E, rows = c["E"], c["rows"]
    share = [(i + 1.0) ** -c["skew"] for i in range(E)]
    total, at, got = sum(share), 0.0, []
    for s in share:
        lo = round(rows * at / total)
        at += s
        got.append(round(rows * at / total) - lo)
    got[-1] += rows - sum(got)
    return got


def work(c):
    op = c["op"]
    if op == "route":
        per = c["E"] * SIZE[c["dtype"]] + c["k"] * 12          # logits; indices, weights, slots
        return {"bytes": c["T"] * per + (c["E"] * 4 if c["bias"] else 0) + 4 * c["E"] + 4, "flops": 4 * c["T"] * c["E"]}
    if op == "quantize":
        out = c["M"] * max(1, c["k"])
        return {"bytes": c["M"] * (c["K"] * SIZE[c["dtype"]] + 4 * c["k"]) + out * (c["K"] + 4 * _cdiv(c["K"], BLOCK)),
                "flops": 3 * c["M"] * c["K"]}
    if op == "swiglu":
        return {"bytes": c["M"] * (2 * c["K"] * SIZE[c["dtype"]] + c["K"] + 4 * _cdiv(c["K"], BLOCK)), "flops": 8 * c["M"] * c["K"]}
    if op == "combine":
        return {"bytes": c["T"] * ((c["k"] + 1) * c["N"] * SIZE[c["dtype"]] + 8 * c["k"]), "flops": 2 * c["T"] * c["k"] * c["N"]}
    KB, NB = _cdiv(c["K"], BLOCK), _cdiv(c["N"], BLOCK)
    rows = c["M"] if op == "gemm" else c["rows"]
    matrices = 1 if op == "gemm" else sum(n > 0 for n in _counts(c))
    return {"bytes": rows * (c["K"] + 4 * KB + c["N"] * SIZE[c["dtype"]]) + matrices * (c["N"] * c["K"] + 4 * NB * KB),
            "flops": 2 * rows * c["N"] * c["K"]}


# -------------------------------------------------------------------------------------------- inputs

def _tokens(shape, g, dtype):
    """Activations as they come out of a norm: Gaussian, a few outlier channels, tokens of unequal size."""
    x = torch.randn(shape, generator=g, device="cuda")
    ch = torch.randint(0, shape[1], (max(1, shape[1] // 512),), generator=g, device="cuda")
    x[:, ch] *= 30.0
    x *= torch.exp(0.5 * torch.randn((shape[0], 1), generator=g, device="cuda"))
    return x.to(dtype)


def _pad(x, dim):
    n = -x.shape[dim] % BLOCK
    if not n:
        return x
    shape = list(x.shape)
    shape[dim] = n
    return torch.cat([x, x.new_zeros(shape)], dim)


def _quantize(x):
    """fp32 [rows, K] -> float8 codes [rows, K], scales [rows, ceil(K / 128)]."""
    rows, K = x.shape
    b = _pad(x, 1).view(rows, -1, BLOCK)
    amax = b.abs().amax(2).clamp_min(TINY)
    codes = (b * (E4M3_MAX / amax)[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(rows, -1)[:, :K].contiguous(), amax / E4M3_MAX


def _weights(N, K, g):
    """One float8 matrix [N, K] of output channels of unequal size, and its 128 x 128 block scales."""
    w = torch.randn((N, K), generator=g, device="cuda") * 0.02
    w *= torch.exp(torch.rand((N, 1), generator=g, device="cuda") * -4.0)
    p = _pad(_pad(w, 0), 1)
    b = p.view(p.shape[0] // BLOCK, BLOCK, -1, BLOCK)
    amax = b.abs().amax((1, 3)).clamp_min(TINY)
    codes = (b * (E4M3_MAX / amax)[:, None, :, None]).to(torch.float8_e4m3fn).view(p.shape)
    return codes[:N, :K].contiguous(), amax / E4M3_MAX


def _slots(T, k, E, g):
    """Rows in expert order for k distinct experts of each token."""
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].contiguous()
    order = torch.argsort(idx.view(-1), stable=True)
    slots = torch.empty(T * k, dtype=torch.int32, device="cuda")
    slots[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    return slots.view(T, k)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    dtype = DTYPES[c["dtype"]]
    op = c["op"]
    if op == "route":
        T, E = c["T"], c["E"]
        logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
        if c["masked"]:      # experts that are switched off, and padding tokens that go nowhere
            logits[:, torch.rand((E,), generator=g, device="cuda") < 0.1] = -math.inf
            logits[torch.rand((T,), generator=g, device="cuda") < 0.05] = -math.inf
        s["logits"] = logits.to(dtype)
        s["bias"] = 0.1 * torch.randn((E,), generator=g, device="cuda") if c["bias"] else None
    elif op == "quantize":
        s["x"] = _tokens((c["M"], c["K"]), g, dtype)
        s["slots"] = _slots(c["M"], c["k"], 64, g) if c["k"] else None
    elif op == "swiglu":
        s["h"] = _tokens((c["M"], 2 * c["K"]), g, dtype)
    elif op == "gemm":
        s["qa"], s["sa"] = _quantize(_tokens((c["M"], c["K"]), g, torch.float32))
        s["qw"], s["sw"] = _weights(c["N"], c["K"], g)
    elif op == "grouped":
        E, N, K = c["E"], c["N"], c["K"]
        s["qa"], s["sa"] = _quantize(_tokens((c["rows"], K), g, torch.float32))
        s["qw"] = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        s["sw"] = torch.empty((E, _cdiv(N, BLOCK), _cdiv(K, BLOCK)), device="cuda")
        for e in range(E):
            s["qw"][e], s["sw"][e] = _weights(N, K, g)
        counts = torch.tensor(_counts(c), device="cuda")[torch.randperm(E, generator=g, device="cuda")]
        s["most"] = max(_counts(c))
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    else:
        T, N, k = c["T"], c["N"], c["k"]
        s["h"] = torch.randn((T * k, N), generator=g, device="cuda").to(dtype)
        s["slots"] = _slots(T, k, 64, g)
        w = torch.rand((T, k), generator=g, device="cuda")
        s["weights"] = w / w.sum(1, keepdim=True)
    return s


# --------------------------------------------------------------------------------------- plain forms

def _route_plain(logits, bias, c):
    """Selection in 64 bits (values next to a border), ties to the lowest index; weights in 32."""
    T, E = logits.shape
    k, G = c["k"], c["n_group"]
    l = logits.double()
    off = torch.isnan(l) | (l == -math.inf)
    l = l.masked_fill(off, -math.inf).clamp_max(torch.finfo(torch.float32).max)
    none = off.all(1, keepdim=True)
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True).masked_fill(none, 0.0))
        p = p / p.sum(1, keepdim=True).masked_fill(none, 1.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    key = l if bias is None else (p + bias.double()).masked_fill(off, -math.inf)
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values
        rank = best[:, :, 0]
        if bias is not None and E // G > 1:
            rank = rank + best[:, :, 1].masked_fill(best[:, :, 1] == -math.inf, 0.0)
        kept = torch.zeros((T, G), dtype=torch.bool, device=key.device)
        kept.scatter_(1, rank.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]], True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    value, idx = key.sort(dim=1, descending=True, stable=True)
    value, idx = value[:, :k], idx[:, :k]
    left = value == -math.inf
    w = p.gather(1, idx).masked_fill(left, 0.0).float()
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return idx.masked_fill(left, -1).to(torch.int32), w * c["scale"]


def _plan_plain(idx, E):
    flat = idx.reshape(-1).long()
    gone = (flat < 0) | (flat >= E)
    key = flat.masked_fill(gone, E)
    order = key.sort(dim=0, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)]).to(torch.int32)
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=idx.device)
    return offsets, slots.masked_fill(gone, -1).to(torch.int32).view(idx.shape)


def _dequantize_rows(q, s):
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _dequantize_weights(q, s):
    full = s.repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)
    return q.float() * full[..., :q.shape[-2], :q.shape[-1]]


def _plain(s, c):
    op = c["op"]
    dtype = DTYPES[c["dtype"]]
    if op == "route":
        idx, w = _route_plain(s["logits"], s["bias"], c)
        offsets, slots = _plan_plain(idx, c["E"])
        return {"idx": idx, "weights": w, "offsets": offsets, "slots": slots}
    if op == "quantize":
        q, sc = _quantize(s["x"].float())
        if s["slots"] is None:
            return {"codes": q, "scales": sc}
        to, k = s["slots"].view(-1).long(), c["k"]
        codes = torch.empty((to.numel(), c["K"]), dtype=torch.uint8, device=q.device)
        scales = torch.empty((to.numel(), sc.shape[1]), device=q.device)
        codes[to] = q.view(torch.uint8).repeat_interleave(k, 0)
        scales[to] = sc.repeat_interleave(k, 0)
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "swiglu":
        gate, up = s["h"].float().split(c["K"], 1)
        q, sc = _quantize(gate / (1.0 + torch.exp(-gate)) * up)
        return {"codes": q, "scales": sc}
    if op == "gemm":
        return (_dequantize_rows(s["qa"], s["sa"]) @ _dequantize_weights(s["qw"], s["sw"]).T).to(dtype)
    if op == "grouped":
        a, off = _dequantize_rows(s["qa"], s["sa"]), s["offsets"].long()
        row = torch.arange(c["rows"], device=a.device)
        e = torch.searchsorted(off[1:], row, right=True)
        at = e * s["most"] + row - off[e]
        padded = a.new_zeros((c["E"] * s["most"], c["K"]))
        padded[at] = a
        y = torch.bmm(padded.view(c["E"], s["most"], c["K"]), _dequantize_weights(s["qw"], s["sw"]).transpose(1, 2))
        return y.view(-1, c["N"])[at].to(dtype)
    return (s["h"].float()[s["slots"].long()] * s["weights"][:, :, None]).sum(1).to(dtype)


def run(state):
    c = state["c"]
    if not own:
        return _plain(state, c)
    import int8_quantized_gemm_gb300 as q8
    op = c["op"]
    if op == "route":
        idx, w = q8.q8_moe_route(state["logits"], c["k"], score=c["score"], bias=state["bias"], n_group=c["n_group"],
                                 topk_group=c["topk_group"], renorm=c["renorm"], scale=c["scale"])
        offsets, slots = q8.q8_moe_plan(idx, c["E"])
        return {"idx": idx, "weights": w, "offsets": offsets, "slots": slots}
    if op == "quantize":
        codes, scales = q8.q8_quantize_fp8(state["x"], slots=state["slots"])
        return {"codes": codes, "scales": scales}
    if op == "swiglu":
        codes, scales = q8.q8_swiglu_quantize_fp8(state["h"])
        return {"codes": codes, "scales": scales}
    if op == "gemm":
        return q8.q8_gemm_fp8(state["qa"], state["sa"], state["qw"], state["sw"], out_dtype=DTYPES[c["dtype"]])
    if op == "grouped":
        return q8.q8_gemm_fp8_grouped(state["qa"], state["sa"], state["qw"], state["sw"], state["offsets"],
                                      out_dtype=DTYPES[c["dtype"]])
    return q8.q8_moe_combine(state["h"], state["slots"], state["weights"])


# ------------------------------------------------------------------------------------------- 64 bits

def _quantize_exact(x):
    """64-bit values -> (what the codes stand for before scaling, scales), block by block."""
    rows, K = x.shape
    codes = torch.empty((rows, K), dtype=torch.float64, device=x.device)
    scales = torch.empty((rows, _cdiv(K, BLOCK)), dtype=torch.float64, device=x.device)
    for b in range(scales.shape[1]):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        scale = torch.maximum(part.max(1).values, -part.min(1).values).clamp_min(TINY) / E4M3_MAX
        codes[:, b * BLOCK:(b + 1) * BLOCK] = (part / scale[:, None]).to(torch.float8_e4m3fn).double()
        scales[:, b] = scale
    return codes, scales


def _product_exact(qa, sa, qw, sw):
    """Block by block along K, in 64 bits."""
    M, K = qa.shape
    y = torch.zeros((M, qw.shape[0]), dtype=torch.float64, device=qa.device)
    channel = torch.arange(qw.shape[0], device=qa.device) // BLOCK
    step = 16 * BLOCK
    for k0 in range(0, K, step):
        at = torch.arange(k0, min(K, k0 + step), device=qa.device) // BLOCK
        a = qa[:, k0:k0 + step].double() * sa.double()[:, at]
        w = qw[:, k0:k0 + step].double() * sw.double()[channel][:, at]
        y.addmm_(a, w.T)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op = c["op"]
    if op == "route":
        l = s["logits"].double().nan_to_num(nan=-math.inf, posinf=torch.finfo(torch.float32).max, neginf=-math.inf)
        p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1).nan_to_num(0.0)
        idx, _ = _route_plain(s["logits"], s["bias"], c)
        w = torch.where(idx >= 0, p.gather(1, idx.long().clamp_min(0)), torch.zeros((), dtype=torch.float64, device="cuda"))
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        return {"idx": None, "weights": w * c["scale"], "offsets": None, "slots": None}
    if op == "quantize":
        codes, scales = _quantize_exact(s["x"].double())
        if s["slots"] is not None:
            token = torch.empty(s["slots"].numel(), dtype=torch.int64, device="cuda")
            token[s["slots"].view(-1).long()] = torch.arange(token.numel(), device="cuda") // c["k"]
            codes, scales = codes[token], scales[token]
        return {"codes": codes, "scales": scales}
    if op == "swiglu":
        h = s["h"].double()
        codes, scales = _quantize_exact(h[:, :c["K"]] * torch.sigmoid(h[:, :c["K"]]) * h[:, c["K"]:])
        return {"codes": codes, "scales": scales}
    if op == "gemm":
        return _product_exact(s["qa"], s["sa"], s["qw"], s["sw"])
    if op == "grouped":
        off = s["offsets"].tolist()
        return torch.cat([_product_exact(s["qa"][off[e]:off[e + 1]], s["sa"][off[e]:off[e + 1]], s["qw"][e], s["sw"][e])
                          for e in range(c["E"])])
    y = torch.zeros((c["T"], c["N"]), dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        y += s["weights"][:, j:j + 1].double() * s["h"][s["slots"][:, j].long()].double()
    return y
