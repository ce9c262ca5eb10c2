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


# ------------------------------------------------------------------------------------------- products

def experts(rows, E, N, K, seed):
    qa, sa = ref.quantize(ref.tokens(rows, K, seed))
    both = [ref.quantize_weight(ref.tokens(N, K, seed + 1 + e) * 0.05) for e in range(E)]
    qw = torch.stack([b[0].view(torch.uint8) for b in both]).view(torch.float8_e4m3fn)
    return [t.cuda() for t in (qa, sa, qw, torch.stack([b[1] for b in both]))]


def test_grouped_work_is_bounded_whatever_the_offsets(q8):
    """Offsets that fall give overlapping ranges, whose rows are not defined; the work for them is that of disjoint ranges
    at most: here 1 + 16 tiles of 16 rows, and the 21st is not computed."""
    E, rows = 40, 16
    offsets = torch.tensor([0, 8] * 20 + [16], dtype=torch.int32)      # every second expert has rows 0 .. 7, the last 8 .. 15
    y = torch.full((rows, 128), 5.0, device="cuda")
    q8.q8_gemm_fp8_grouped(*experts(rows, E, 128, 256, 1), offsets.cuda(), out_dtype=torch.float32, out=y)
    assert (y[8:] == 5).all() and (y[:8] != 5).any()
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("rows,N,K", [(600, 520, 528), (1300, 1100, 1040), (300, 136, 2064)])
def test_grouped_overlapping_ranges_end(q8, rows, N, K):
    """The same for many rows an expert: the call ends, and a disjoint call after it is right."""
    args = experts(rows, 4, N, K, 2)
    y = torch.full((rows, N), 5.0, device="cuda")
    overlapping = torch.tensor([0, rows, 0, rows, rows // 2], dtype=torch.int32, device="cuda")
    q8.q8_gemm_fp8_grouped(*args, overlapping, out_dtype=torch.float32, out=y)
    offsets = torch.tensor([0, rows // 3, rows // 3, rows - 7, rows], dtype=torch.int32)
    q8.q8_gemm_fp8_grouped(*args, offsets.cuda(), out_dtype=torch.float32, out=y)
    qa, sa, qw, sw = (t.cpu() for t in args)
    for e in (0, 2, 3):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        want, mag = ref.product(qa[at], sa[at], qw[e], sw[e])
        assert ((y[at].cpu().double() - want).abs() <= ref.product_tolerance(want, mag, K, torch.float32)).all()
    assert q8.q8_device_error() == 0
