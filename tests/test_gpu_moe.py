"""Routing, the experts' rows and the weighted sum against plain forms in 64 bits; the whole layer and its capture."""
import math

import pytest
import torch

from . import fp8_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def q8():
    import int8_quantized_gemm_gb300 as q8
    return q8


def check_route(q8, logits, k, bias=None, **how):
    idx, w = q8.q8_moe_route(logits.cuda(), k, bias=None if bias is None else bias.cuda(), **how)
    want_idx, want_w = ref.route(logits, k, bias=bias, **dict({"score": "softmax"}, **how))
    assert torch.equal(idx.cpu(), want_idx)
    # the score: exp (2 steps), the rounding of its argument (|l - m| below 90: 90 half steps of a score that is
    # then e^-90; at most 0.4 of the largest), a sum of up to 512 terms in 5 + E / 32 additions, two divisions
    E = logits.shape[1]
    tol = (2.0 ** -24) * (2 * (8 + E / 32 + 8)) * want_w.abs().amax(1, keepdim=True).clamp_min(1e-30)
    assert ((w.cpu().double() - want_w).abs() <= tol + 1e-37).all()
    return idx, w


CASES = [
    # T, E, k, n_group, topk_group
    (1, 8, 1, 1, 1), (1, 256, 8, 8, 4), (5, 16, 16, 1, 1), (33, 64, 6, 1, 1), (17, 100, 7, 1, 1), (40, 96, 5, 3, 2),
    (9, 512, 8, 1, 1), (20, 160, 6, 8, 3), (12, 32, 32, 32, 32), (7, 510, 9, 17, 5), (3, 2, 1, 2, 1), (129, 33, 3, 1, 1),
    (6, 448, 20, 7, 7), (30, 1, 1, 1, 1),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_route(q8, i, with_bias, score):
    T, E, k, n_group, topk_group = CASES[i]
    g = torch.Generator().manual_seed(i)
    logits = torch.randn((T, E), generator=g).to(DTYPES[i % 3])
    bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
    check_route(q8, logits, k, bias, score=score, n_group=n_group, topk_group=topk_group, renorm=i % 2 == 0,
                scale=1.0 if i % 3 else 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1), (4, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_ties_and_masks(q8, score, groups, with_bias):
    """Few distinct logits (ties to the lowest index), masked experts, rows with one or no expert left, NaN, +inf,
    and the type's lowest value, which is a number and not a mask."""
    g = torch.Generator().manual_seed(11)
    logits = torch.randint(-2, 3, (64, 32), generator=g).to(torch.bfloat16)
    logits[torch.rand((64, 32), generator=g) < 0.3] = -math.inf
    logits[0] = -math.inf
    logits[1] = math.nan
    logits[2] = -math.inf
    logits[2, 17] = 1.0
    logits[3] = torch.finfo(torch.bfloat16).min
    logits[4, 5] = math.inf
    logits[5, 7] = math.nan
    logits[6] = 0.0
    logits[6, ::2] = -0.0
    bias = torch.zeros(32) if with_bias else None
    if with_bias:
        bias[::5] = 0.25
    check_route(q8, logits, 6, bias, score=score, n_group=groups[0], topk_group=groups[1], renorm=True, scale=1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_near_ties_are_decided_in_64_bits(q8, score):
    """Keys nearer than fp32 tells apart: score + bias equal to 1e-9 by construction."""
    g = torch.Generator().manual_seed(2)
    T, E = 50, 64
    logits = torch.randn((T, E), generator=g)
    for t in range(T):                                   # neighbours with logits one fp32 step apart
        logits[t, 1::2] = torch.nextafter(logits[t, ::2], torch.tensor(math.inf if t % 2 else -math.inf))
    bias = torch.randn(E // 2, generator=g).repeat_interleave(2) * 0.05
    check_route(q8, logits, 8, bias, score=score, renorm=True, scale=1.0)
    check_route(q8, logits, 8, bias, score=score, n_group=8, topk_group=3, renorm=True, scale=1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_too_few_experts_and_masking_bias(q8, score):
    """One group of four cannot give six experts; a bias of -inf or NaN masks, +inf puts first; equal keys throughout."""
    g = torch.Generator().manual_seed(5)
    logits = torch.randn((40, 32), generator=g)
    bias = torch.zeros(32)
    idx, w = check_route(q8, logits, 6, bias, score=score, n_group=8, topk_group=1)
    assert (idx[:, 4:] == -1).all() and (w[:, 4:] == 0).all()
    bias[3], bias[7], bias[11], bias[30] = -math.inf, math.nan, math.inf, -math.inf
    check_route(q8, logits, 6, bias, score=score)
    check_route(q8, logits, 31, bias, score=score, renorm=False)
    check_route(q8, torch.zeros(9, 32), 30, bias, score=score)         # every key equal, more than 28 left: -1
    check_route(q8, torch.zeros(9, 32), 5, bias, score=score, n_group=4, topk_group=2)


def test_route_all_equal_over_lanes(q8):
    """512 equal keys: the first experts, through the fp64 path with more candidates than lanes."""
    for bias in (None, torch.zeros(512)):
        check_route(q8, torch.full((3, 512), 0.25), 32, bias, score="sigmoid")


def test_route_strided_rows(q8):
    base = torch.randn((21, 100), generator=torch.Generator().manual_seed(1)).cuda()
    x = base[::3, 5:69]
    idx, w = q8.q8_moe_route(x, 4)
    want, _ = ref.route(x.cpu(), 4, "softmax")
    assert torch.equal(idx.cpu(), want)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (7, 3, 5), (130, 8, 64), (1031, 6, 160), (4096, 8, 512),
                                   (20001, 2, 3), (9000, 8, 128)])
def test_plan(q8, T, k, E):
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(-1, E + (1 if T % 2 else 0), (T, k), generator=g).to(torch.int32)
    offsets, slots = q8.q8_moe_plan(idx.cuda(), E)
    want_o, want_s = ref.plan(idx, E)
    assert torch.equal(offsets.cpu(), want_o) and torch.equal(slots.cpu(), want_s)


def test_plan_extremes(q8):
    offsets, slots = q8.q8_moe_plan(torch.full((300, 4), -1, dtype=torch.int32, device="cuda"), 8)
    assert (offsets == 0).all() and (slots == -1).all()
    idx = torch.full((5000, 1), 3, dtype=torch.int32, device="cuda")
    offsets, slots = q8.q8_moe_plan(idx, 8)
    assert offsets.tolist() == [0, 0, 0, 0, 5000, 5000, 5000, 5000, 5000]
    assert torch.equal(slots.view(-1).cpu(), torch.arange(5000, dtype=torch.int32))
    offsets, slots = q8.q8_moe_plan(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 8)
    assert (offsets == 0).all() and slots.shape == (0, 4)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N,k", [(1, 8, 1), (3, 136, 5), (65, 1024, 8), (17, 4096, 2), (10, 64, 32)])
def test_combine(q8, dtype, T, N, k):
    g = torch.Generator().manual_seed(N)
    rows = T * k + 2
    h = torch.randn((rows, N), generator=g).to(dtype)
    slots = torch.randperm(rows, generator=g)[:T * k].to(torch.int32).view(T, k)
    w = torch.rand((T, k), generator=g)
    slots[torch.rand((T, k), generator=g) < 0.2] = -1
    slots[T // 2] = -1                                   # a token that went nowhere
    if T > 2:
        slots[0, 0] = rows                               # outside: adds nothing
    y = q8.q8_moe_combine(h.cuda(), slots.cuda(), w.cuda()).cpu().double()
    in_ = (slots >= 0) & (slots < rows)
    terms = h.double()[slots.clamp(0, rows - 1).long()] * (w.double() * in_)[:, :, None]
    want, mag = terms.sum(1), terms.abs().sum(1)
    sums = k * 2.0 ** -24 * mag
    assert ((y - want).abs() <= sums + ref.EPS[dtype] * (want.abs() + sums) + 2.0 ** -25 * (dtype == torch.float16)).all()
    assert (y[T // 2] == 0).all()


# -------------------------------------------------------------------------------------------- the layer

def layer(q8, x, logits, bias, w13, w2, k, E):
    idx, w = q8.q8_moe_route(logits, k, score="sigmoid", bias=bias, scale=2.0)
    offsets, slots = q8.q8_moe_plan(idx, E)
    qa, sa = q8.q8_quantize_fp8(x, slots=slots)
    h = q8.q8_gemm_fp8_grouped(qa, sa, *w13, offsets)
    qh, sh = q8.q8_swiglu_quantize_fp8(h)
    return q8.q8_moe_combine(q8.q8_gemm_fp8_grouped(qh, sh, *w2, offsets), slots, w), idx, w


@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_layer_and_its_capture(q8, T):
    """The calls of one layer of routed experts against the layer in 64 bits on the dequantized weights, then captured
    in a graph and replayed on other inputs."""
    E, k, H, I = 16, 4, 512, 256
    g = torch.Generator().manual_seed(T)
    x = [torch.randn((T, H), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    logits = [torch.randn((T, E), generator=g).cuda() for _ in range(2)]
    bias = (0.1 * torch.randn(E, generator=g)).cuda()
    w13 = q8.q8_quantize_weight_fp8((torch.randn((E, 2 * I, H), generator=g) * H ** -0.5).cuda())
    w2 = q8.q8_quantize_weight_fp8((torch.randn((E, H, I), generator=g) * I ** -0.5).cuda())
    eager = [layer(q8, a, b, bias, w13, w2, k, E) for a, b in zip(x, logits)]
    for (y, idx, w), a in zip(eager, x):
        d13 = torch.stack([ref.values(w13[0][e].cpu(), w13[1][e].cpu(), weight=True) for e in range(E)])
        d2 = torch.stack([ref.values(w2[0][e].cpu(), w2[1][e].cpu(), weight=True) for e in range(E)])
        want = torch.zeros((T, H), dtype=torch.float64)
        for t in range(T):
            for e, p in zip(idx[t].tolist(), w[t].double().tolist()):
                h = d13[e] @ a[t].cpu().double()
                want[t] += p * (d2[e] @ (h[:I] / (1 + torch.exp(-h[:I])) * h[I:]))
        # two roundings to e4m3 (half a step, 2^-4 of a value, on either side of the gate's product), uncorrelated
        # over 256 and 512 terms: under 2^-4 of the result's norm
        assert (y.cpu().double() - want).norm() <= 2.0 ** -4 * want.norm()
    sx, sl = x[0].clone(), logits[0].clone()
    layer(q8, sx, sl, bias, w13, w2, k, E)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, _ = layer(q8, sx, sl, bias, w13, w2, k, E)
    for i in (1, 0):
        sx.copy_(x[i])
        sl.copy_(logits[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i][0])
    assert q8.q8_device_error() == 0


def test_results_belong_to_the_stream_that_writes_them(q8):
    """Results allocated by a call with a stream come from that stream's memory."""
    side = torch.cuda.Stream()
    logits = torch.randn((64, 16), device="cuda")
    torch.cuda.synchronize()
    idx, w = q8.q8_moe_route(logits, 2, stream=side)
    offsets, slots = q8.q8_moe_plan(idx, 16, stream=side)
    side.synchronize()
    want, _ = ref.route(logits.cpu(), 2, "softmax")
    assert torch.equal(idx.cpu(), want)
    wo, ws = ref.plan(want, 16)
    assert torch.equal(offsets.cpu(), wo) and torch.equal(slots.cpu(), ws)


def test_example_runs_small():
    """examples/moe_layer.py on a small layer with sizes that are no multiple of a tile."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst = example.main(["--experts", "12", "--top-k", "3", "--hidden", "528", "--inter", "272", "--tokens", "1,7,130"])
    assert worst < 2.0 ** -4
