"""Plain 64-bit (and, where the operator is defined bit by bit, fp32) forms of the float8 and
routed-expert operators for the tests. CPU tensors; no code of the package."""
import math

import torch

BLOCK, FP8_MAX, TINY = 128, 448.0, 1e-30
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative


def cdiv(a, b):
    return -(-a // b)


def quantize(x):
    """The definition in fp32, operation by operation: codes and scales of fp32 [rows, K]."""
    rows, K = x.shape
    KB = cdiv(K, BLOCK)
    q = torch.empty((rows, K), dtype=torch.float8_e4m3fn)
    s = torch.empty((rows, KB), dtype=torch.float32)
    for b in range(KB):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        a = part.abs().amax(1)                    # propagates NaN
        a = torch.where(a < TINY, torch.tensor(TINY), a)
        s[:, b] = a / torch.tensor(FP8_MAX)
        q[:, b * BLOCK:(b + 1) * BLOCK] = (part * (torch.tensor(FP8_MAX) / a)[:, None]).to(torch.float8_e4m3fn)
    return q, s


def quantize_weight(w):
    """The same over 128 x 128 blocks of fp32 [N, K]."""
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.float8_e4m3fn)
    s = torch.empty((cdiv(N, BLOCK), cdiv(K, BLOCK)), dtype=torch.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            a = w[at].abs().max()
            a = torch.tensor(TINY) if a < TINY else a
            s[i, j] = a / torch.tensor(FP8_MAX)
            q[at] = (w[at] * (torch.tensor(FP8_MAX) / a)).to(torch.float8_e4m3fn)
    return q, s


def values(q, s, weight=False):
    """What the codes stand for, in 64 bits."""
    full = s.double().repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]
    if weight:
        full = full.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :]
    return q.double() * full


def product(qa, sa, qw, sw):
    """(y, sum of the products' magnitudes) in 64 bits."""
    a, w = values(qa, sa), values(qw, sw, weight=True)
    return a @ w.T, a.abs() @ w.abs().T


def product_tolerance(y, mag, K, dtype):
    """fp32 sums of up to 128 products (a step of the sum per addition, whichever way the tensor core
    rounds), one rounded multiply-add a block with a rounded scale product, one rounding to dtype."""
    sums = (BLOCK + cdiv(K, BLOCK) + 4) * 2.0 ** -23 * mag
    floor = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -149      # half a step of the subnormals
    return sums + EPS[dtype] * (y.abs() + sums) + floor


def route(logits, k, score, bias=None, n_group=1, topk_group=1, renorm=True, scale=1.0):
    """idx int32 and 64-bit weights."""
    T, E = logits.shape
    l = logits.double()
    off = torch.isnan(l) | (l == -math.inf)
    l = torch.where(off, torch.tensor(-math.inf, dtype=torch.float64), l.clamp_max(3.4028234663852886e38))
    idx = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        live = [e for e in range(E) if not off[t, e]]
        if not live:
            continue
        if score == "softmax":
            m = max(float(l[t, e]) for e in live)
            z = sum(math.exp(float(l[t, e]) - m) for e in live)
            p = {e: math.exp(float(l[t, e]) - m) / z for e in live}
        else:
            p = {e: (1.0 / (1.0 + math.exp(-float(l[t, e]))) if float(l[t, e]) > -700 else 0.0) for e in live}
        key = {e: (float(l[t, e]) if bias is None else p[e] + float(bias[e])) for e in live}
        key = {e: v for e, v in key.items() if v > -math.inf}      # nor NaN: a bias can mask too
        if n_group > 1:
            per = E // n_group
            rank = []
            for g in range(n_group):
                own = sorted((key[e] for e in range(g * per, (g + 1) * per) if e in key), reverse=True)
                if own:
                    rank.append((-(own[0] if bias is None or len(own) == 1 else own[0] + own[1]), g))
            kept = {g for _, g in sorted(rank)[:topk_group]}
            key = {e: v for e, v in key.items() if e // per in kept}
        best = sorted(key, key=lambda e: (-key[e], e))[:k]
        for j, e in enumerate(best):
            idx[t, j], w[t, j] = e, p[e]
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp_min(1e-300), torch.zeros_like(w))
    return idx, w * scale


def plan(idx, E):
    T, k = idx.shape
    flat = idx.reshape(-1).tolist()
    counts = [0] * E
    for e in flat:
        if 0 <= e < E:
            counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    at, slots = offsets[:], []
    for e in flat:
        if 0 <= e < E:
            slots.append(at[e])
            at[e] += 1
        else:
            slots.append(-1)
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(slots, dtype=torch.int32).view(T, k)


def tokens(rows, K, seed, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, K), generator=g)
    if outliers:
        x[:, torch.randint(0, K, (max(1, K // 256),), generator=g)] *= 30.0
    return x
