"""Refusals of the float8 and routed-expert entry points: validation runs before any CUDA call, so these need no GPU
(the pointers are never read). Also the reference forms the GPU tests compare with, on values known by hand."""
import ctypes
import math

import pytest
import torch

from . import fp8_reference as ref

P = ctypes.c_void_p
FAKE, ODD = P(0x10000), P(0x10002)
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    from int8_quantized_gemm_gb300 import build
    build.build()
    import int8_quantized_gemm_gb300 as q8
    return q8.load()


OK, INVALID, UNSUPPORTED = 0, 1, 2


def call(lib, name, defaults, **change):
    args = dict(defaults, **change)
    if name == "q8_moe_route":
        args["scale"] = ctypes.c_float(args["scale"])
    return getattr(lib, name)(*args.values(), None)


QUANT = dict(x=FAKE, type=0, M=4, K=128, ldx=128, slots=None, top_k=0, rows_out=4, q=FAKE, s=FAKE)
SWIGLU = dict(h=FAKE, type=1, M=4, I=128, ldh=256, q=FAKE, s=FAKE)
WEIGHT = dict(w=FAKE, type=0, E=2, N=128, K=128, qw=FAKE, sw=FAKE)
GEMM = dict(qa=FAKE, sa=FAKE, qw=FAKE, sw=FAKE, M=4, N=8, K=128, y=FAKE, type=0)
GROUPED = dict(qa=FAKE, sa=FAKE, qw=FAKE, sw=FAKE, offsets=FAKE, rows=4, E=2, N=8, K=128, y=FAKE, type=0)
ROUTE = dict(logits=FAKE, type=0, T=4, E=16, ldl=16, top_k=2, score=0, bias=None, n_group=1, topk_group=1, renorm=1,
             scale=1.0, idx=FAKE, weights=FAKE)
PLAN = dict(idx=FAKE, T=4, top_k=2, E=16, offsets=FAKE, slots=FAKE)
COMBINE = dict(h=FAKE, type=1, rows=8, N=64, slots=FAKE, weights=FAKE, T=4, top_k=2, y=FAKE)

REFUSED = [
    ("q8_quantize_fp8", QUANT, dict(x=None), INVALID),
    ("q8_quantize_fp8", QUANT, dict(x=ODD), INVALID),
    ("q8_quantize_fp8", QUANT, dict(q=None), INVALID),
    ("q8_quantize_fp8", QUANT, dict(s=None), INVALID),
    ("q8_quantize_fp8", QUANT, dict(type=3), INVALID),
    ("q8_quantize_fp8", QUANT, dict(M=-1, rows_out=-1), INVALID),
    ("q8_quantize_fp8", QUANT, dict(ldx=127), INVALID),
    ("q8_quantize_fp8", QUANT, dict(rows_out=5), INVALID),
    ("q8_quantize_fp8", QUANT, dict(top_k=1), INVALID),
    ("q8_quantize_fp8", QUANT, dict(slots=FAKE, top_k=0), INVALID),
    ("q8_quantize_fp8", QUANT, dict(slots=ODD, top_k=1), INVALID),
    ("q8_quantize_fp8", QUANT, dict(slots=FAKE, top_k=33), UNSUPPORTED),
    ("q8_quantize_fp8", QUANT, dict(K=120, ldx=120), UNSUPPORTED),
    ("q8_quantize_fp8", QUANT, dict(ldx=130), UNSUPPORTED),
    ("q8_quantize_fp8", QUANT, dict(type=1, ldx=132), UNSUPPORTED),
    ("q8_quantize_fp8", QUANT, dict(M=BIG, rows_out=BIG), UNSUPPORTED),
    ("q8_swiglu_quantize_fp8", SWIGLU, dict(h=None), INVALID),
    ("q8_swiglu_quantize_fp8", SWIGLU, dict(ldh=255), INVALID),
    ("q8_swiglu_quantize_fp8", SWIGLU, dict(I=-16), INVALID),
    ("q8_swiglu_quantize_fp8", SWIGLU, dict(I=24, ldh=48), UNSUPPORTED),
    ("q8_quantize_weight_fp8", WEIGHT, dict(w=None), INVALID),
    ("q8_quantize_weight_fp8", WEIGHT, dict(E=-1), INVALID),
    ("q8_quantize_weight_fp8", WEIGHT, dict(K=24), UNSUPPORTED),
    ("q8_quantize_weight_fp8", WEIGHT, dict(qw=ODD), INVALID),
    ("q8_gemm_fp8", GEMM, dict(qa=None), INVALID),
    ("q8_gemm_fp8", GEMM, dict(sa=None), INVALID),
    ("q8_gemm_fp8", GEMM, dict(qw=ODD), INVALID),
    ("q8_gemm_fp8", GEMM, dict(y=None), INVALID),
    ("q8_gemm_fp8", GEMM, dict(y=ODD), INVALID),
    ("q8_gemm_fp8", GEMM, dict(type=-1), INVALID),
    ("q8_gemm_fp8", GEMM, dict(M=-1), INVALID),
    ("q8_gemm_fp8", GEMM, dict(K=100), UNSUPPORTED),
    ("q8_gemm_fp8", GEMM, dict(M=BIG), UNSUPPORTED),
    ("q8_gemm_fp8", GEMM, dict(N=BIG), UNSUPPORTED),
    ("q8_gemm_fp8_grouped", GROUPED, dict(offsets=None), INVALID),
    ("q8_gemm_fp8_grouped", GROUPED, dict(offsets=ODD), INVALID),
    ("q8_gemm_fp8_grouped", GROUPED, dict(E=513), UNSUPPORTED),
    ("q8_gemm_fp8_grouped", GROUPED, dict(E=512, N=1 << 23), UNSUPPORTED),
    ("q8_gemm_fp8_grouped", GROUPED, dict(K=0), UNSUPPORTED),
    ("q8_gemm_fp8_grouped", GROUPED, dict(sw=None), INVALID),
    ("q8_moe_route", ROUTE, dict(logits=None), INVALID),
    ("q8_moe_route", ROUTE, dict(idx=None), INVALID),
    ("q8_moe_route", ROUTE, dict(score=2), INVALID),
    ("q8_moe_route", ROUTE, dict(top_k=17), INVALID),
    ("q8_moe_route", ROUTE, dict(top_k=0), INVALID),
    ("q8_moe_route", ROUTE, dict(n_group=3), INVALID),
    ("q8_moe_route", ROUTE, dict(n_group=4, topk_group=5), INVALID),
    ("q8_moe_route", ROUTE, dict(ldl=15), INVALID),
    ("q8_moe_route", ROUTE, dict(scale=math.inf), INVALID),
    ("q8_moe_route", ROUTE, dict(E=513, ldl=513), UNSUPPORTED),
    ("q8_moe_route", ROUTE, dict(E=64, ldl=64, top_k=33), UNSUPPORTED),
    ("q8_moe_route", ROUTE, dict(E=66, ldl=66, n_group=33), UNSUPPORTED),
    ("q8_moe_plan", PLAN, dict(idx=None), INVALID),
    ("q8_moe_plan", PLAN, dict(offsets=None), INVALID),
    ("q8_moe_plan", PLAN, dict(E=0), INVALID),
    ("q8_moe_plan", PLAN, dict(E=513), UNSUPPORTED),
    ("q8_moe_plan", PLAN, dict(T=1 << 30, top_k=2), UNSUPPORTED),
    ("q8_moe_combine", COMBINE, dict(h=None), INVALID),
    ("q8_moe_combine", COMBINE, dict(y=ODD), INVALID),
    ("q8_moe_combine", COMBINE, dict(N=63), UNSUPPORTED),
    ("q8_moe_combine", COMBINE, dict(top_k=33), UNSUPPORTED),
    ("q8_moe_combine", COMBINE, dict(rows=-1), INVALID),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refused(lib, i):
    name, defaults, change, status = REFUSED[i]
    assert call(lib, name, defaults, **change) == status, (name, change)


EMPTY = [
    ("q8_quantize_fp8", QUANT, dict(M=0, rows_out=0, x=None, q=None, s=None)),
    ("q8_quantize_fp8", QUANT, dict(K=0, ldx=0)),
    ("q8_swiglu_quantize_fp8", SWIGLU, dict(M=0, h=None, q=None, s=None)),
    ("q8_quantize_weight_fp8", WEIGHT, dict(E=0, w=None, qw=None, sw=None)),
    ("q8_gemm_fp8", GEMM, dict(M=0)),
    ("q8_gemm_fp8", GEMM, dict(N=0)),
    ("q8_gemm_fp8_grouped", GROUPED, dict(rows=0, qa=None, sa=None, y=None)),
    ("q8_gemm_fp8_grouped", GROUPED, dict(E=0)),
    ("q8_moe_route", ROUTE, dict(T=0, logits=None, idx=None, weights=None)),
    ("q8_moe_combine", COMBINE, dict(T=0, h=None, slots=None, weights=None, y=None)),
]


@pytest.mark.parametrize("i", range(len(EMPTY)))
def test_empty_problems_enqueue_nothing(lib, i):
    name, defaults, change = EMPTY[i]
    before = lib.q8_launch_count()
    assert call(lib, name, defaults, **change) == OK
    assert lib.q8_launch_count() == before


def test_binding_refuses_cpu_tensors_and_shapes():
    import int8_quantized_gemm_gb300 as q8
    x = torch.zeros(4, 128)
    for call in (lambda: q8.q8_quantize_fp8(x), lambda: q8.q8_swiglu_quantize_fp8(x),
                 lambda: q8.q8_quantize_weight_fp8(x), lambda: q8.q8_gemm_fp8(x, x, x, x),
                 lambda: q8.q8_gemm_fp8_grouped(x, x, x, x, x), lambda: q8.q8_moe_route(x, 1),
                 lambda: q8.q8_moe_plan(x, 4), lambda: q8.q8_moe_combine(x, x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        q8.q8_quantize_weight_fp8(x.int())
    with pytest.raises(TypeError):
        q8.q8_moe_route([1.0], 1)


def test_reference_quantizer_by_hand():
    x = torch.zeros(3, 144)
    x[0, 0], x[0, 1], x[0, 130] = 448.0, 17.0, -2.0
    x[1, 3] = math.inf
    q, s = ref.quantize(x)
    assert s[0, 0] == 1.0 and q[0, 0].item() == 448.0
    assert q[0, 1].item() == 16.0                    # a tie between 16 and 18 goes to the even code
    assert q[0, 130].item() == -448.0 and s[0, 1] == torch.tensor(2.0) / torch.tensor(448.0)
    assert torch.isnan(ref.values(q, s)[1, :128]).all() and (ref.values(q, s)[1, 128:] == 0).all()
    assert (q[2].float() == 0).all() and (s[2] > 0).all()


def test_reference_route_by_hand():
    l = torch.tensor([[1.0, 3.0, 3.0, -math.inf], [-math.inf] * 4, [0.0, math.nan, -1.0, -math.inf]])
    idx, w = ref.route(l, 2, "softmax")
    assert idx.tolist() == [[1, 2], [-1, -1], [0, 2]]
    assert w[1].tolist() == [0.0, 0.0] and abs(w[0, 0].item() - 0.5) < 1e-12
    idx, _ = ref.route(l, 3, "sigmoid", bias=torch.tensor([0.9, 0.0, 0.0, 0.0]))
    assert idx.tolist() == [[0, 1, 2], [-1, -1, -1], [0, 2, -1]]
    idx, _ = ref.route(torch.tensor([[5.0, 0.0, 4.0, 3.9]]), 2, "sigmoid", bias=torch.zeros(4), n_group=2, topk_group=1)
    assert idx.tolist() == [[2, 3]]                  # a pair of good experts beats the one best
    offsets, slots = ref.plan(torch.tensor([[1, 0], [-1, 1], [7, 1]], dtype=torch.int32), 2)
    assert offsets.tolist() == [0, 1, 4] and slots.tolist() == [[1, 0], [-1, 2], [-1, 3]]
