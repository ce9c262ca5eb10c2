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


# ------------------------------------------------------------------------------- results, slots

def pool_stream(t):
    """The stream whose memory pool of PyTorch's allocator the tensor lies in."""
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= t.data_ptr() < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not memory of the allocator")


def test_results_are_allocated_for_the_stream_that_writes_them(q8):
    """A result's memory comes from the pool of the call's stream: from another's, it could be handed out again to work that
    is not ordered after the call."""
    def calls(stream):
        x = torch.randn((40, 256), device="cuda").to(torch.bfloat16)
        logits = torch.randn((40, 8), device="cuda")
        w = torch.randn((8, 256, 256), device="cuda")
        torch.cuda.synchronize()
        kept = [x, logits, w]
        idx, weights = q8.q8_moe_route(logits, 2, stream=stream)
        offsets, slots = q8.q8_moe_plan(idx, 8, stream=stream)
        qw, sw = q8.q8_quantize_weight_fp8(w, stream=stream)
        qa, sa = q8.q8_quantize_fp8(x, slots=slots, stream=stream)
        qd, sd = q8.q8_quantize_fp8(x, stream=stream)
        h = q8.q8_gemm_fp8_grouped(qa, sa, qw, sw, offsets, stream=stream)
        y = q8.q8_gemm_fp8(qd, sd, qw[0], sw[0], stream=stream)
        qh, sh = q8.q8_swiglu_quantize_fp8(h, stream=stream)
        out = q8.q8_moe_combine(h, slots, weights, stream=stream)
        torch.cuda.synchronize()
        return kept, (idx, weights, offsets, slots, qw, sw, qa, sa, qd, sd, h, y, qh, sh, out)

    side = torch.cuda.Stream()
    kept, results = calls(side)
    assert {pool_stream(t) for t in results} == {side.cuda_stream}
    assert side.cuda_stream not in {pool_stream(t) for t in kept}
    kept, results = calls(None)
    assert {pool_stream(t) for t in results} == {pool_stream(kept[0])} != {side.cuda_stream}


@pytest.mark.parametrize("M,K,k", [(1, 16, 32), (9, 400, 3), (70, 2064, 8)])
def test_quantize_fp16_to_slots(q8, M, K, k):
    """Every slot of a row holds the row's codes and scales, bit for bit."""
    x = ref.tokens(M, K, seed=M).to(torch.float16)
    slots = torch.randperm(M * k, generator=torch.Generator().manual_seed(M)).to(torch.int32).view(M, k)
    q, s = q8.q8_quantize_fp8(x.cuda(), slots=slots.cuda())
    wq, ws = ref.quantize(x.float())
    for j in range(k):
        at = slots[:, j].long()
        assert torch.equal(q.view(torch.uint8).cpu()[at], wq.view(torch.uint8)) and torch.equal(s.cpu()[at], ws)


def test_slots_that_are_no_matrix_of_indices(q8):
    x = torch.zeros((4, 128), device="cuda")
    one = torch.zeros(4, dtype=torch.int32, device="cuda")
    for slots, error in (([0, 1, 2, 3], TypeError), (one, ValueError), (one[0], ValueError), (one.view(4, 1).long(), TypeError),
                         (one.view(4, 1).cpu(), ValueError), (one.view(2, 2), ValueError)):
        with pytest.raises(error):
            q8.q8_quantize_fp8(x, slots=slots)
