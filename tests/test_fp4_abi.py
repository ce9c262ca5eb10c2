"""Refusals of the 4-bit floating-point entry points: validation runs before any CUDA call, so these need no GPU (the pointers
are never read). Also the reference forms the GPU tests compare with, on values known by hand."""
import math

import pytest
import torch

from . import fp4_reference as ref
from .test_fp8_abi import BIG, FAKE, INVALID, ODD, OK, UNSUPPORTED, call, lib  # noqa: F401  (lib is the fixture)

QUANT = dict(x=FAKE, type=0, block=16, M=4, K=128, ldx=128, slots=None, top_k=0, rows_out=4, q=FAKE, sf=FAKE, s=FAKE)
SWIGLU = dict(h=FAKE, type=1, block=32, M=4, I=128, ldh=256, q=FAKE, sf=FAKE, s=None)
WEIGHT = dict(w=FAKE, type=0, block=16, E=2, N=128, K=128, qw=FAKE, sfw=FAKE, sw=FAKE)
BACK = dict(q=FAKE, sf=FAKE, s=FAKE, block=16, rows=4, K=128, tile_rows=0, y=FAKE, type=1)
GEMM = dict(qa=FAKE, sfa=FAKE, sa=FAKE, qw=FAKE, sfw=FAKE, sw=FAKE, block=16, M=4, N=8, K=128, y=FAKE, type=0)
GROUPED = dict(qa=FAKE, sfa=FAKE, sa=FAKE, qw=FAKE, sfw=FAKE, sw=FAKE, offsets=FAKE, block=32, rows=4, E=2, N=8, K=128, y=FAKE,
               type=0)

REFUSED = [
    ("q8_quantize_fp4", QUANT, dict(x=None), INVALID),
    ("q8_quantize_fp4", QUANT, dict(x=ODD), INVALID),
    ("q8_quantize_fp4", QUANT, dict(q=None), INVALID),
    ("q8_quantize_fp4", QUANT, dict(sf=None), INVALID),
    ("q8_quantize_fp4", QUANT, dict(sf=ODD), INVALID),
    ("q8_quantize_fp4", QUANT, dict(s=None), INVALID),
    ("q8_quantize_fp4", QUANT, dict(type=3), INVALID),
    ("q8_quantize_fp4", QUANT, dict(block=8), INVALID),
    ("q8_quantize_fp4", QUANT, dict(block=0), INVALID),
    ("q8_quantize_fp4", QUANT, dict(M=-1, rows_out=-1), INVALID),
    ("q8_quantize_fp4", QUANT, dict(ldx=127), INVALID),
    ("q8_quantize_fp4", QUANT, dict(rows_out=5), INVALID),
    ("q8_quantize_fp4", QUANT, dict(top_k=1), INVALID),
    ("q8_quantize_fp4", QUANT, dict(slots=FAKE, top_k=0), INVALID),
    ("q8_quantize_fp4", QUANT, dict(slots=ODD, top_k=1), INVALID),
    ("q8_quantize_fp4", QUANT, dict(slots=FAKE, top_k=33), UNSUPPORTED),
    ("q8_quantize_fp4", QUANT, dict(K=112, ldx=112), UNSUPPORTED),
    ("q8_quantize_fp4", QUANT, dict(ldx=130), UNSUPPORTED),
    ("q8_quantize_fp4", QUANT, dict(M=BIG, rows_out=BIG), UNSUPPORTED),
    ("q8_quantize_fp4", QUANT, dict(K=BIG, ldx=BIG), UNSUPPORTED),
    ("q8_swiglu_quantize_fp4", SWIGLU, dict(h=None), INVALID),
    ("q8_swiglu_quantize_fp4", SWIGLU, dict(block=16), INVALID),       # without row scales
    ("q8_swiglu_quantize_fp4", SWIGLU, dict(ldh=255), INVALID),
    ("q8_swiglu_quantize_fp4", SWIGLU, dict(I=-32), INVALID),
    ("q8_swiglu_quantize_fp4", SWIGLU, dict(I=48, ldh=96), UNSUPPORTED),
    ("q8_quantize_weight_fp4", WEIGHT, dict(w=None), INVALID),
    ("q8_quantize_weight_fp4", WEIGHT, dict(E=-1), INVALID),
    ("q8_quantize_weight_fp4", WEIGHT, dict(sw=None), INVALID),
    ("q8_quantize_weight_fp4", WEIGHT, dict(block=64), INVALID),
    ("q8_quantize_weight_fp4", WEIGHT, dict(K=48), UNSUPPORTED),
    ("q8_quantize_weight_fp4", WEIGHT, dict(qw=ODD), INVALID),
    ("q8_quantize_weight_fp4", WEIGHT, dict(E=1 << 20, N=1 << 21), UNSUPPORTED),
    ("q8_dequantize_fp4", BACK, dict(q=None), INVALID),
    ("q8_dequantize_fp4", BACK, dict(y=ODD), INVALID),
    ("q8_dequantize_fp4", BACK, dict(s=ODD), INVALID),
    ("q8_dequantize_fp4", BACK, dict(type=4), INVALID),
    ("q8_dequantize_fp4", BACK, dict(type=3), INVALID),                # float8 holds no scaled values
    ("q8_dequantize_fp4", BACK, dict(block=1), INVALID),
    ("q8_dequantize_fp4", BACK, dict(tile_rows=3), INVALID),
    ("q8_dequantize_fp4", BACK, dict(K=16), UNSUPPORTED),
    ("q8_dequantize_fp4", BACK, dict(rows=1 << 39, K=1 << 20), UNSUPPORTED),
    ("q8_gemm_fp4", GEMM, dict(qa=None), INVALID),
    ("q8_gemm_fp4", GEMM, dict(sfa=None), INVALID),
    ("q8_gemm_fp4", GEMM, dict(sfw=ODD), INVALID),
    ("q8_gemm_fp4", GEMM, dict(sa=ODD), INVALID),
    ("q8_gemm_fp4", GEMM, dict(qw=ODD), INVALID),
    ("q8_gemm_fp4", GEMM, dict(y=None), INVALID),
    ("q8_gemm_fp4", GEMM, dict(y=ODD), INVALID),
    ("q8_gemm_fp4", GEMM, dict(type=3), INVALID),
    ("q8_gemm_fp4", GEMM, dict(block=128), INVALID),
    ("q8_gemm_fp4", GEMM, dict(M=-1), INVALID),
    ("q8_gemm_fp4", GEMM, dict(K=144), UNSUPPORTED),
    ("q8_gemm_fp4", GEMM, dict(M=BIG), UNSUPPORTED),
    ("q8_gemm_fp4", GEMM, dict(M=BIG - 200), UNSUPPORTED),
    ("q8_gemm_fp4", GEMM, dict(N=BIG - 1), UNSUPPORTED),
    ("q8_gemm_fp4", GEMM, dict(K=BIG - 256), UNSUPPORTED),
    ("q8_gemm_fp4", GEMM, dict(N=1 << 24, K=1 << 18), UNSUPPORTED),    # tiles of scales past 32 bits
    ("q8_gemm_fp4_grouped", GROUPED, dict(offsets=None), INVALID),
    ("q8_gemm_fp4_grouped", GROUPED, dict(offsets=ODD), INVALID),
    ("q8_gemm_fp4_grouped", GROUPED, dict(E=513), UNSUPPORTED),
    ("q8_gemm_fp4_grouped", GROUPED, dict(E=512, N=1 << 23), UNSUPPORTED),
    ("q8_gemm_fp4_grouped", GROUPED, dict(K=0), UNSUPPORTED),
    ("q8_gemm_fp4_grouped", GROUPED, dict(rows=BIG - 16), UNSUPPORTED),
]


@pytest.mark.parametrize("name,defaults,change,status", REFUSED)
def test_refused(lib, name, defaults, change, status):  # noqa: F811
    assert call(lib, name, defaults, **change) == status


@pytest.mark.parametrize("name,defaults,change", [
    ("q8_quantize_fp4", QUANT, dict(M=0, rows_out=0, x=None, q=None, sf=None, s=None)),
    ("q8_quantize_fp4", QUANT, dict(M=0, rows_out=7, top_k=3, x=None)),
    ("q8_quantize_fp4", QUANT, dict(K=0, ldx=0, x=None)),
    ("q8_swiglu_quantize_fp4", SWIGLU, dict(I=0, ldh=0, h=None)),
    ("q8_quantize_weight_fp4", WEIGHT, dict(E=0, w=None)),
    ("q8_dequantize_fp4", BACK, dict(rows=0, q=None)),
    ("q8_gemm_fp4", GEMM, dict(M=0, qa=None, y=None)),
    ("q8_gemm_fp4", GEMM, dict(N=0, qw=None, y=None)),
    ("q8_gemm_fp4_grouped", GROUPED, dict(rows=0, offsets=None, qa=None)),
    ("q8_gemm_fp4_grouped", GROUPED, dict(E=0, offsets=None, qw=None)),
])
def test_nothing_to_do(lib, name, defaults, change):  # noqa: F811
    assert call(lib, name, defaults, **change) == OK


def test_binding_refuses_what_is_on_the_host():
    import int8_quantized_gemm_gb300 as q8
    x = torch.zeros((4, 64))
    for f in (q8.q8_quantize_fp4, q8.q8_swiglu_quantize_fp4):
        with pytest.raises(ValueError, match="CUDA"):
            f(x)
    for f in (q8.q8_quantize_weight_fp4, q8.q8_dequantize_fp4):
        with pytest.raises((TypeError, ValueError)):
            f(x)
    for bad in (None, 3, x, x.int()):
        with pytest.raises((TypeError, ValueError)):
            q8.q8_quantize_fp4(bad)
        with pytest.raises((TypeError, ValueError)):
            q8.q8_gemm_fp4(bad, bad, None, bad, bad, None)
        with pytest.raises((TypeError, ValueError)):
            q8.q8_dequantize_fp4(bad)


# ------------------------------------------------------------------------------- the reference, by hand

def test_reference_levels():
    t = torch.tensor([0.0, 0.25, 0.26, 0.74, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.1, 100.0, -0.25, -0.3, -5.0])
    want = [0, 0, 1, 1, 2, 2, 3, 4, 4, 5, 6, 6, 7, 7, 8, 9, 14]
    assert ref.e2m1(t).tolist() == want
    assert torch.equal(ref.e2m1(ref.LEVELS), torch.arange(16, dtype=torch.uint8))


def test_reference_block32():
    x = torch.zeros((1, 128))
    x[0, 0], x[0, 33], x[0, 64] = 6.0, 6.1, -1.5
    codes, sf, s = ref.quantize(x, 32)
    assert s is None and sf[0].tolist() == [127, 128, 125, 0]
    assert codes[0, 0] == 7 and codes[0, 33] == 5 and codes[0, 64] == 15      # 6, 3.05 -> 3, -6
    assert float(ref.values(codes, sf, s, 32)[0, 64]) == -1.5


def test_reference_block16():
    x = torch.zeros((2, 64))
    x[0, 0], x[0, 16], x[0, 40] = 2688.0, 6.0, -3.0
    x[1, 5] = math.inf
    codes, sf, s = ref.quantize(x, 16)
    assert float(s[0]) == 1.0 and torch.isnan(s[1])
    c = ref.scale_values(sf, 16)[0].tolist()
    assert c == [448.0, 1.0, 0.5, 0.0]
    v = ref.values(codes, sf, s, 16)[0]
    assert float(v[0]) == 2688.0 and float(v[16]) == 6.0 and float(v[40]) == -3.0 and float(v.abs().sum()) == 2697.0


def test_reference_layout():
    sf = torch.arange(200 * 18, dtype=torch.int64).remainder(251).to(torch.uint8).view(200, 18)     # K = 288, blocks of 16
    t = ref.tile(sf, 288, 16)
    assert t.shape == (2, 8, 32, 4, 4)
    assert int(t[1, 4, 7, 2, 1]) == int(sf[128 + 2 * 32 + 7, 17])
    assert int(t[1, 0, 8, 2, 0]) == 0 and int(t[0, 4, 0, 0, 2]) == 0                                # no row 200, no block 18
    q = ref.pack(torch.tensor([[1, 15, 7, 8]], dtype=torch.uint8))
    assert q.tolist() == [[0xF1, 0x87]] and ref.unpack(q).tolist() == [[1, 15, 7, 8]]
