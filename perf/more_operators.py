"""Workloads of the 4-bit floating-point operators: what is measured, and their plain forms.

The cases are the steps of a linear layer, and of a layer of routed experts, with weights and activations of
4-bit e2m1 codes: quantizing the tokens (also into expert order), the gated activation, the product, and the experts'
products, from one token to prefill batches. Two microscaled formats: a scale for each 16 K in e4m3 under one fp32 scale a
row (block 16), and a power of two for each 32 K (block 32). `run` computes a step in elementary torch operations
(own = False) or through the package's entry points (own = True).
"""
import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)       # what the codes 0..7 stand for; bit 3 is the sign
E4M3_MAX = 448.0
ROW_MAX = 6.0 * E4M3_MAX                                # a row's largest value, in units of its scale
TINY = 1e-30                                            # the smallest row maximum a scale is made from
SPAN = 256                                              # rows of scales are padded to whole spans of 256 K
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def _cdiv(a, b):
    return -(-a // b)


def _pitch(K, block):
    return _cdiv(K, SPAN) * (SPAN // block)


# --------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token: launch latency
        dict(name="quantize 1x8192", op="quantize", M=1, K=8192, k=0, block=16, dtype="bf16"),
        # the activations of the int8 prefill16k layer, quantized to 4 bits instead
        dict(name="quantize 8192x16384", op="quantize", M=8192, K=16384, k=0, block=16, dtype="fp32"),
        # an odd batch of tokens written once into each of its experts' slots
        dict(name="quantize 1037x4096 to 8 slots", op="quantize", M=1037, K=4096, k=8, block=32, dtype="bf16"),
        # the gated activation of a decode batch of 16 tokens with 8 experts each
        dict(name="swiglu 128x2048", op="swiglu", M=128, K=2048, block=32, dtype="fp16"),
        # and of a prefill batch of 4096 tokens
        dict(name="swiglu 32768x2048", op="swiglu", M=32768, K=2048, block=16, dtype="bf16"),
        # the decode layer of the framework's own benchmark, with 4-bit weights
        dict(name="gemm 16x28672x8192", op="gemm", M=16, N=28672, K=8192, block=16, dtype="bf16"),
        # a ragged shape: no dimension is a multiple of a tile, the last span of scales is short
        dict(name="gemm 517x2056x4128", op="gemm", M=517, N=2056, K=4128, block=32, dtype="fp32"),
        # a batch between decode and prefill
        dict(name="gemm 256x8192x8192", op="gemm", M=256, N=8192, K=8192, block=16, dtype="fp16"),
        # the prefill layer of the framework's own benchmark
        dict(name="gemm 8192x8192x16384", op="gemm", M=8192, N=8192, K=16384, block=16, dtype="bf16"),
        # a decode batch of 16 tokens to 8 of 64 experts: every active expert's weights are read for a few rows
        dict(name="experts 128 rows of 64", op="grouped", rows=128, E=64, N=4096, K=4096, skew=0.5, block=32, dtype="bf16"),
        # an odd batch in between: some tens of rows an expert
        dict(name="experts 2050 rows of 32", op="grouped", rows=2050, E=32, N=4096, K=2048, skew=0.5, block=16, dtype="fp16"),
        # a prefill batch of 4096 tokens to 8 of 64 experts, unevenly spread
        dict(name="experts 32768 rows of 64", op="grouped", rows=32768, E=64, N=4096, K=4096, skew=0.5, block=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "swiglu", "gemm", "gemm", "gemm", "gemm", "grouped", "grouped", "grouped"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    block = rng.choice([16, 32])
    if op == "quantize":
        k = rng.choice([0, 0, 1, 4, 8])
        K = 32 * _log(rng, 2, 512)
        return dict(op=op, M=_log(rng, 1, min(32768, (1 << 27) // (K * max(1, k)))), K=K, k=k, block=block, dtype=dtype)
    if op == "swiglu":
        K = 32 * _log(rng, 2, 256)
        return dict(op=op, M=_log(rng, 1, min(65536, (1 << 26) // K)), K=K, block=block, dtype=dtype)
    if op == "gemm":
        K = 32 * _log(rng, 4, 512)
        N = _log(rng, 64, min(28672, (1 << 28) // K))
        return dict(op=op, M=_log(rng, 1, min(8192, (1 << 39) // (N * K))), N=N, K=K, block=block, dtype=dtype)
    E = _log(rng, 2, 128)
    K = 32 * _log(rng, 8, 128)
    N = _log(rng, 64, min(8192, (1 << 30) // (E * K)))
    return dict(op=op, rows=_log(rng, 1, min(32768, (1 << 38) // (N * K))), E=E, N=N, K=K, skew=rng.choice([0.0, 0.5, 1.0]),
                block=block, dtype=dtype)


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
    op, K, block = c["op"], c["K"], c["block"]
    row = K // 2 + K // block + (4 if block == 16 else 0)         # codes, scales and the row's scale
    if op in ("quantize", "swiglu"):
        # the tokens in; the codes, the scales; the codes read again and written as values
        out = c["M"] * max(1, c.get("k", 0))
        read = K * SIZE[c["dtype"]] * (2 if op == "swiglu" else 1) + 4 * c.get("k", 0)
        return {"bytes": c["M"] * read + out * (row + K // 2 + K), "flops": (8 if op == "swiglu" else 3) * c["M"] * K}
    rows = c["M"] if op == "gemm" else c["rows"]
    matrices = 1 if op == "gemm" else sum(n > 0 for n in _counts(c))
    return {"bytes": rows * (row + c["N"] * SIZE[c["dtype"]]) + matrices * c["N"] * row, "flops": 2 * rows * c["N"] * K}


# ------------------------------------------------------------------------------------------ plain forms

def _quantize(x, block):
    """fp32 [rows, K] -> codes uint8 [rows, K], scales [rows, K / block] in their own type, row scales (block 16)."""
    rows, K = x.shape
    b = x.view(rows, K // block, block)
    amax = b.abs().amax(2)
    if block == 16:
        top = amax.amax(1).clamp_min(TINY)
        s = top / ROW_MAX
        sf = (amax * (E4M3_MAX / top)[:, None]).to(torch.float8_e4m3fn)
        f = sf.float()
        up = torch.where(f > 0, (ROW_MAX / top)[:, None] / f, torch.zeros_like(f))
    else:       # the smallest power of two that keeps the block within 6
        s = None
        m, e = torch.frexp(amax)                                 # amax = m 2^e, m in [1/2, 1)
        e = torch.where(m <= 0.75, e - 3, e - 2).clamp_min(-127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        sf = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        up = torch.ldexp(torch.ones_like(amax), -e)
    t = (b * up[:, :, None]).view(rows, K)
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]            # halfway: to the even code
    borders[1::2] = [float(torch.nextafter(torch.tensor(v), torch.tensor(0.0))) for v in borders[1::2]]
    code = torch.bucketize(t.abs(), torch.tensor(borders, device=x.device), out_int32=True)
    return (code + 8 * (t < 0)).to(torch.uint8), sf, s


def _values(codes):
    """What codes stand for, before any scale."""
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    return lut[codes.int()]


def _pad_scales(sf, K, block):
    n = _pitch(K, block) - sf.shape[-1]
    raw = sf.view(torch.uint8)
    return torch.cat([raw, raw.new_zeros((*raw.shape[:-1], n))], -1).view(sf.dtype) if n else sf


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpack(q):
    return torch.stack([q & 15, q >> 4], -1).view(*q.shape[:-1], 2 * q.shape[-1])


def _tile(sf, K, block):
    """Scales [N, K / block] of a weight matrix in tiles of 128 rows x 4 scales, [N / 128, ., 32, 4, 4]: the scale g of row n is at
    [n / 128, g / 4, n % 32, n % 128 / 32, g % 4]; zeros where there is no row or no K."""
    raw = _pad_scales(sf, K, block).view(torch.uint8)
    n = -raw.shape[0] % 128
    raw = torch.cat([raw, raw.new_zeros((n, raw.shape[1]))])
    t = raw.view(raw.shape[0] // 128, 4, 32, raw.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return t.contiguous().view(sf.dtype)


def _untile(sf, N, K, block):
    """The way back, for one matrix or several: fp32 [..., N, K / block]."""
    t = sf.view(torch.uint8).movedim(-2, -4).movedim(-2, -3)      # [..., N / 128, 4, 32, ., 4]
    raw = t.reshape(*sf.shape[:-5], sf.shape[-5] * 128, sf.shape[-4] * 4)[..., :N, :K // block]
    return raw.contiguous().view(sf.dtype).float()


def _dequantize(q, sf, s, block):
    """fp32 values of packed codes [..., K / 2] with scales [..., K / block] and row scales."""
    v = _values(_unpack(q)) * sf.repeat_interleave(block, -1)
    return v if s is None else v * s[..., None]


def _plain(s, c):
    op, K, block = c["op"], c["K"], c["block"]
    dtype = DTYPES[c["dtype"]]
    if op in ("quantize", "swiglu"):
        if op == "quantize":
            x = s["x"].float()
        else:
            gate, up = s["h"].float().split(K, 1)
            x = gate / (1.0 + torch.exp(-gate)) * up
        codes, sf, row = _quantize(x.contiguous(), block)
        values, sf = _values(codes).to(torch.float8_e4m3fn), _pad_scales(sf, K, block)
        if s.get("slots") is not None:
            to, k = s["slots"].view(-1).long(), c["k"]
            token = torch.empty_like(to)
            token[to] = torch.arange(to.numel(), device=to.device) // k
            values = values.view(torch.uint8)[token].view(torch.float8_e4m3fn)
            sf = sf.view(torch.uint8)[token].view(sf.dtype)
            row = None if row is None else row[token]
        return {"codes": values, "scales": sf} if row is None else {"codes": values, "scales": sf, "rows": row}
    a = _dequantize(s["qa"], s["sfa"][:, :K // block].float(), s["sa"], block)
    w = _dequantize(s["qw"], _untile(s["sfw"], c["N"], K, block), s["sw"], block)
    if op == "gemm":
        return (a @ w.T).to(dtype)
    off = s["offsets"].long()
    row = torch.arange(c["rows"], device=a.device)
    e = torch.searchsorted(off[1:], row, right=True)
    at = e * s["most"] + row - off[e]
    padded = a.new_zeros((c["E"] * s["most"], K))
    padded[at] = a
    y = torch.bmm(padded.view(c["E"], s["most"], K), w.transpose(1, 2))
    return y.view(-1, c["N"])[at].to(dtype)


# -------------------------------------------------------------------------------------------- inputs

def _tokens(shape, g, dtype):
    """Activations as they come out of a norm: Gaussian, a few outlier channels, tokens of unequal size."""
    x = torch.randn(shape, generator=g, device="cuda")
    ch = torch.randint(0, shape[1], (max(1, shape[1] // 512),), generator=g, device="cuda")
    x[:, ch] *= 30.0
    x *= torch.exp(0.5 * torch.randn((shape[0], 1), generator=g, device="cuda"))
    return x.to(dtype)


def _weights(N, K, block, g):
    """One 4-bit matrix [N, K] of output channels of unequal size: packed codes, tiled scales, channel scales."""
    w = torch.randn((N, K), generator=g, device="cuda") * 0.02
    w *= torch.exp(torch.rand((N, 1), generator=g, device="cuda") * -4.0)
    codes, sf, s = _quantize(w, block)
    return _pack(codes), _tile(sf, K, block), s


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
    dtype, op, K, block = DTYPES[c["dtype"]], c["op"], c["K"], c["block"]
    if op == "quantize":
        s["x"] = _tokens((c["M"], K), g, dtype)
        s["slots"] = _slots(c["M"], c["k"], 64, g) if c["k"] else None
        return s
    if op == "swiglu":
        s["h"] = _tokens((c["M"], 2 * K), g, dtype)
        return s
    codes, sfa, s["sa"] = _quantize(_tokens((c["M"] if op == "gemm" else c["rows"], K), g, torch.float32), block)
    s["qa"], s["sfa"] = _pack(codes), _pad_scales(sfa, K, block)
    if op == "gemm":
        s["qw"], s["sfw"], s["sw"] = _weights(c["N"], K, block, g)
        return s
    got = [_weights(c["N"], K, block, g) for _ in range(c["E"])]
    s["qw"] = torch.stack([w[0] for w in got])
    s["sfw"] = torch.stack([w[1].view(torch.uint8) for w in got]).view(got[0][1].dtype)
    s["sw"] = torch.stack([w[2] for w in got]) if block == 16 else None
    counts = torch.tensor(_counts(c), device="cuda")[torch.randperm(c["E"], generator=g, device="cuda")]
    s["most"] = max(_counts(c))
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return s


def run(state):
    c = state["c"]
    if not own:
        return _plain(state, c)
    import int8_quantized_gemm_gb300 as q8
    op, block = c["op"], c["block"]
    if op in ("quantize", "swiglu"):
        if op == "quantize":
            q, sf, row = q8.q8_quantize_fp4(state["x"], block=block, slots=state["slots"])
        else:
            q, sf, row = q8.q8_swiglu_quantize_fp4(state["h"], block=block)
        values = q8.q8_dequantize_fp4(q, out_dtype=torch.float8_e4m3fn)
        return {"codes": values, "scales": sf} if row is None else {"codes": values, "scales": sf, "rows": row}
    a, w = (state["qa"], state["sfa"], state["sa"]), (state["qw"], state["sfw"], state["sw"])
    if op == "gemm":
        return q8.q8_gemm_fp4(*a, *w, out_dtype=DTYPES[c["dtype"]])
    return q8.q8_gemm_fp4_grouped(*a, *w, state["offsets"], out_dtype=DTYPES[c["dtype"]])


# ------------------------------------------------------------------------------------------- 64 bits

def _quantize_exact(x, block):
    """64-bit values -> (what the codes stand for before scaling, scales padded, row scales)."""
    rows, K = x.shape
    amax = torch.maximum(x.view(rows, -1, block).max(2).values, -x.view(rows, -1, block).min(2).values)
    row = None
    if block == 16:
        row = amax.max(1).values.clamp_min(TINY) / (6.0 * E4M3_MAX)
        sf = (amax / 6.0 / row[:, None]).to(torch.float8_e4m3fn).double()
        unit = sf * row[:, None]
    else:
        sf = torch.exp2(torch.ceil(torch.log2(amax.clamp_min(2.0 ** -140) / 6.0)).clamp_min(-127.0))
        unit = sf
    t = x / unit.clamp_min(1e-300).repeat_interleave(block, 1)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(1e-300))).clamp(0.0, 2.0) - 1.0)
    codes = (torch.round(t / step) * step).clamp(-6.0, 6.0)
    codes[(unit == 0).repeat_interleave(block, 1)] = 0.0
    pad = torch.full((rows, _pitch(K, block) - sf.shape[1]), 0.0 if block == 16 else 2.0 ** -127, dtype=torch.float64,
                     device=x.device)
    return codes, torch.cat([sf, pad], 1), row


def _weight_values(q, sf, s, N, K, block):
    """64-bit [N, K], tile by tile of scales."""
    lut = torch.tensor([sign * v for sign in (1.0, -1.0) for v in LEVELS], dtype=torch.float64, device=q.device)
    w = torch.empty((N, K), dtype=torch.float64, device=q.device)
    w[:, 0::2], w[:, 1::2] = lut[(q & 15).int()], lut[(q >> 4).int()]
    n, k = torch.arange(N, device=q.device), torch.arange(K // block, device=q.device)
    scale = sf.float()[n[:, None] // 128, k // 4, n[:, None] % 32, n[:, None] % 128 // 32, k % 4].double()
    if s is not None:
        scale = scale * s.double()[:, None]
    return w.mul_(scale.repeat_interleave(block, 1))


def _row_values(q, sf, s, block):
    lut = torch.tensor([sign * v for sign in (1.0, -1.0) for v in LEVELS], dtype=torch.float64, device=q.device)
    a = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    a[:, 0::2], a[:, 1::2] = lut[(q & 15).int()], lut[(q >> 4).int()]
    scale = sf.float().double()[:, :a.shape[1] // block].repeat_interleave(block, 1)
    return a * scale if s is None else a * scale * s.double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op, K, block = c["op"], c["K"], c["block"]
    if op in ("quantize", "swiglu"):
        if op == "quantize":
            x = s["x"].double()
        else:
            h = s["h"].double()
            x = h[:, :K] * torch.sigmoid(h[:, :K]) * h[:, K:]
        codes, sf, row = _quantize_exact(x, block)
        if s.get("slots") is not None:
            token = torch.empty(s["slots"].numel(), dtype=torch.int64, device="cuda")
            token[s["slots"].view(-1).long()] = torch.arange(token.numel(), device="cuda") // c["k"]
            codes, sf, row = codes[token], sf[token], None if row is None else row[token]
        return {"codes": codes, "scales": sf} if row is None else {"codes": codes, "scales": sf, "rows": row}
    a = _row_values(s["qa"], s["sfa"], s["sa"], block)
    if op == "gemm":
        return a @ _weight_values(s["qw"], s["sfw"], s["sw"], c["N"], K, block).T
    off = s["offsets"].tolist()
    return torch.cat([a[off[e]:off[e + 1]] @ _weight_values(s["qw"][e], s["sfw"][e], None if s["sw"] is None else s["sw"][e],
                                                            c["N"], K, block).T for e in range(c["E"])])
