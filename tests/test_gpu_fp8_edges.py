"""Float8 quantizers and products at the edges of their definition, against plain forms in 64 bits."""
import pytest
import torch

from . import fp8_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def q8():
    import int8_quantized_gemm_gb300 as q8
    yield q8
    torch.cuda.synchronize()
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lo,hi,size", [(-4.0, 4.0, 1.0), (-20.0, -1.0, 1.0), (-40.0, -20.0, 1.0), (-60.0, -40.0, 1e4),
                                        (-80.0, -60.0, 6e4), (-87.0, -80.0, 3e30), (-103.0, -87.0, 3e34)])
def test_swiglu_of_closed_gates(q8, dtype, lo, hi, size):
    """Gates of one range a block. Off by 2^-20 of the value (an exponential 2^-21, its sum with 1, three more products or
    sums half a step each, a reciprocal 2^-23, the scale's division: 15 2^-24), and where exp(-|g|) is not a normal
    number by its two steps of 2^-149 times |g u|."""
    if dtype == torch.float16:
        size = min(size, 6e4)
    M, I = 24, 272
    g = torch.Generator().manual_seed(int(-lo))
    gate = (lo + (hi - lo) * torch.rand((M, I), generator=g)).to(dtype)
    up = (torch.randn((M, I), generator=g).clamp(-1, 1) * size).to(dtype)
    q, s = q8.q8_swiglu_quantize_fp8(torch.cat([gate, up], 1).cuda())
    gate, up = gate.double(), up.double()
    x = gate / (1.0 + torch.exp(-gate)) * up
    off = 2.0 ** -20 * x.abs() + 2.0 ** -148 * (gate * up).abs() * (gate < -87.3) + 2.0 ** -149
    for b in range(s.shape[1]):
        at = slice(b * 128, (b + 1) * 128)
        a = x[:, at].abs().amax(1)
        err = (s[:, b].cpu().double() * 448.0 - a.clamp_min(1e-30)).abs()
        assert (err <= off[:, at].amax(1) + 2.0 ** -23 * a.clamp_min(1e-30)).all(), (err / a).max().item()
    sc = s.cpu().double().repeat_interleave(128, 1)[:, :I]
    v, t = q.cpu().double(), x / sc
    half = torch.maximum(t.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
    assert ((v - t).abs() <= half * (1 + 2.0 ** -10) + off / sc + t.abs() * 2.0 ** -20).all()
