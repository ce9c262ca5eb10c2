"""Float8 quantizers and products against plain forms: the quantizers bit for bit (they are defined in fp32
operations), the products against 64 bits within the bound of their fp32 sums and one output rounding."""
import math

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


def same_codes(got, want):
    got, want = got.cpu().float(), want.float()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


def same_scales(got, want):
    got = got.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(posinf=1.0), want.nan_to_num(posinf=1.0))


# ----------------------------------------------------------------------------------------- quantizers

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (5, 1040), (64, 4096), (257, 272), (2, 16384)])
def test_quantize(q8, dtype, M, K):
    x = ref.tokens(M, K, seed=M + K).to(dtype)
    q, s = q8.q8_quantize_fp8(x.cuda())
    wq, ws = ref.quantize(x.float())
    same_codes(q, wq)
    same_scales(s, ws)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_extremes(q8, dtype):
    """Zero blocks, subnormals, the type's largest value, infinities and NaN: a broken value breaks its own block only."""
    x = ref.tokens(8, 400, seed=3).to(dtype)
    x[0] = 0.0
    x[1, :] = torch.finfo(dtype).tiny
    x[2, 5] = torch.finfo(dtype).max
    x[3, 130] = math.inf
    x[4, 399] = -math.inf
    x[5, 128] = math.nan
    x[6, 0], x[6, 1] = math.nan, math.inf
    x[7] = -0.0
    q, s = q8.q8_quantize_fp8(x.cuda())
    wq, ws = ref.quantize(x.float())
    same_codes(q, wq)
    same_scales(s, ws)
    v = ref.values(q.cpu(), s.cpu())
    assert torch.isnan(v[3, 128:256]).all() and torch.isfinite(v[3, :128]).all() and torch.isfinite(v[3, 256:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_strided_rows(q8, dtype):
    base = ref.tokens(33, 512, seed=5).to(dtype).cuda()
    x = base[::2, 64:64 + 272]
    q, s = q8.q8_quantize_fp8(x)
    wq, ws = ref.quantize(x.float().cpu())
    same_codes(q, wq)
    same_scales(s, ws)
    with pytest.raises(ValueError):
        q8.q8_quantize_fp8(base.t())
    with pytest.raises(q8.Q8Error):
        q8.q8_quantize_fp8(base[:, 1:1 + 272])       # rows are not 16-byte aligned


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,k", [(1, 128, 1), (7, 400, 3), (65, 1024, 8)])
def test_quantize_to_slots(q8, dtype, M, K, k):
    """Rows go to their slots; slots outside the result are skipped and rows that nobody has stay."""
    x = ref.tokens(M, K, seed=M).to(dtype)
    g = torch.Generator().manual_seed(M)
    rows = M * k + 3
    slots = torch.randperm(rows, generator=g)[:M * k].to(torch.int32).view(M, k)
    slots[torch.rand((M, k), generator=g) < 0.2] = -1
    if M > 1:
        slots[0, 0] = rows                            # outside: skipped
    KB = ref.cdiv(K, 128)
    q = torch.full((rows, K), 2.0, device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((rows, KB), 7.0, device="cuda")
    q8.q8_quantize_fp8(x.cuda(), slots=slots.cuda(), rows=rows, q=q, s=s)
    wq, ws = ref.quantize(x.float())
    want_q, want_s = torch.full((rows, K), 2.0), torch.full((rows, KB), 7.0)
    for m in range(M):
        for d in slots[m].tolist():
            if 0 <= d < rows:
                want_q[d], want_s[d] = wq[m].float(), ws[m]
    same_codes(q, want_q)
    same_scales(s, want_s)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,I", [(1, 16), (3, 144), (130, 1040), (33, 2048)])
def test_swiglu_quantize(q8, dtype, M, I):
    """Scales within the activation's fp32 error, 2^-19; codes within one step where that moves a value over a
    rounding border, which a relative error of 2^-19 does for about 2^-19 / 2^-4 of them."""
    h = ref.tokens(M, 2 * I, seed=I, outliers=False).to(dtype)
    q, s = q8.q8_swiglu_quantize_fp8(h.cuda())
    g, u = h[:, :I].double(), h[:, I:].double()
    x = g / (1.0 + torch.exp(-g)) * u
    for b in range(s.shape[1]):
        a = x[:, b * 128:(b + 1) * 128].abs().amax(1).clamp_min(1e-30)
        assert ((s[:, b].cpu().double() - a / 448.0).abs() <= 2.0 ** -19 * a / 448.0).all()
    v, sc = q.cpu().double(), s.cpu().double().repeat_interleave(128, 1)[:, :I]
    t = x / sc                                                       # the value before rounding to e4m3
    half = torch.maximum(t.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))   # half a step, or a subnormal's
    assert ((v - t).abs() <= half * (1 + 2.0 ** -10) + t.abs() * 2.0 ** -19).all()


def test_swiglu_strided_and_extremes(q8):
    base = ref.tokens(9, 1024, seed=1, outliers=False).to(torch.bfloat16)
    base[1, 0], base[2, 3], base[3, 260] = math.nan, math.inf, -math.inf
    base[4, 0], base[4, 256] = -3e38, 1.0                            # silu of a very negative gate is -0
    h = base.cuda()[:, :512]
    q, s = q8.q8_swiglu_quantize_fp8(h)
    v = ref.values(q.cpu(), s.cpu())
    assert torch.isnan(v[1, :128]).all() and torch.isnan(v[2, :128]).all() and torch.isnan(v[3, :128]).all()
    assert torch.isfinite(v[1:4, 128:]).all() and torch.isfinite(v[4]).all() and v[4, 0] == 0
    assert torch.isfinite(v[0]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (1, 128, 128), (3, 130, 272), (2, 257, 1040)])
def test_quantize_weight(q8, dtype, E, N, K):
    w = (ref.tokens(E * N, K, seed=N) * 0.02).to(dtype).view(E, N, K)
    qw, sw = q8.q8_quantize_weight_fp8(w.cuda())
    for e in range(E):
        wq, ws = ref.quantize_weight(w[e].float())
        same_codes(qw[e], wq)
        same_scales(sw[e], ws)
    if E == 1:
        q2, s2 = q8.q8_quantize_weight_fp8(w[0].cuda())
        assert torch.equal(q2.view(torch.uint8), qw[0].view(torch.uint8)) and torch.equal(s2, sw[0])


# ------------------------------------------------------------------------------------------- products

def operands(M, N, K, seed, E=None):
    qa, sa = ref.quantize(ref.tokens(M, K, seed))
    if E is None:
        qw, sw = ref.quantize_weight(ref.tokens(N, K, seed + 1) * 0.05)
    else:
        both = [ref.quantize_weight(ref.tokens(N, K, seed + 1 + e) * 0.05) for e in range(E)]
        qw = torch.stack([b[0].view(torch.uint8) for b in both]).view(torch.float8_e4m3fn)
        sw = torch.stack([b[1] for b in both])
    return qa, sa, qw, sw


def check(y, qa, sa, qw, sw, dtype):
    want, mag = ref.product(qa, sa, qw, sw)
    tol = ref.product_tolerance(want, mag, qa.shape[1], dtype)
    err = (y.cpu().double() - want).abs()
    assert (err <= tol).all(), f"largest error over tolerance: {(err / tol).max().item()}"


SHAPES = [(1, 128, 128), (1, 8, 16), (1, 1, 1040), (2, 130, 144), (15, 257, 512), (16, 2056, 4112), (17, 128, 2048),
          (33, 640, 1040), (64, 256, 4096), (65, 136, 256), (128, 384, 640), (129, 264, 400), (256, 256, 1024),
          (300, 520, 528), (517, 1032, 784), (1000, 96, 2064), (2500, 1500, 400), (400, 1500, 2064),
          (300, 200, 16), (600, 521, 128), (70, 201, 112), (2500, 1503, 272),
          (2500, 1503, 4112), (2500, 1502, 4112), (517, 1030, 4112), (1400, 1031, 4112)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(q8, M, N, K):
    dtype = DTYPES[(M + N) % 3]
    qa, sa, qw, sw = operands(M, N, K, seed=M)
    y = q8.q8_gemm_fp8(qa.cuda(), sa.cuda(), qw.cuda(), sw.cuda(), out_dtype=dtype)
    check(y, qa, sa, qw, sw, dtype)


@pytest.mark.parametrize("M,N,K", [(1, 20480, 512), (3, 28672, 1024), (4, 11000, 2048), (5, 30000, 256), (40, 20000, 512)])
def test_gemm_few_tokens_many_tiles(q8, M, N, K):
    """Several tiles for each cluster, K shared by its CTAs, some of which own no token's sum (tokens go round in fours)."""
    qa, sa, qw, sw = operands(M, 128, K, seed=M)
    copies = ref.cdiv(N, 128)
    qw = qw.view(torch.uint8).repeat(copies, 1)[:N].view(qw.dtype)
    sw = sw.repeat(copies, 1) * (1.0 + torch.arange(copies)[:, None] % 7)
    for _ in range(3):
        y = q8.q8_gemm_fp8(qa.cuda(), sa.cuda(), qw.cuda(), sw.cuda(), out_dtype=torch.float32)
    check(y, qa, sa, qw, sw, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(3, 200, 384), (200, 300, 384), (700, 515, 640)])
def test_gemm_types_and_repeats(q8, dtype, M, N, K):
    qa, sa, qw, sw = operands(M, N, K, seed=N)
    dev = [t.cuda() for t in (qa, sa, qw, sw)]
    y = q8.q8_gemm_fp8(*dev, out_dtype=dtype)
    check(y, qa, sa, qw, sw, dtype)
    for _ in range(3):
        assert torch.equal(q8.q8_gemm_fp8(*dev, out_dtype=dtype), y)


def test_gemm_unequal_scales(q8):
    """Scales over 12 orders of magnitude: each block's partial sum gets its own."""
    M, N, K = 40, 300, 1040
    qa, sa, qw, sw = operands(M, N, K, seed=9)
    g = torch.Generator().manual_seed(1)
    sa = sa * torch.exp(14 * (torch.rand(sa.shape, generator=g) - 0.5))
    sw = sw * torch.exp(14 * (torch.rand(sw.shape, generator=g) - 0.5))
    y = q8.q8_gemm_fp8(qa.cuda(), sa.cuda(), qw.cuda(), sw.cuda(), out_dtype=torch.float32)
    check(y, qa, sa, qw, sw, torch.float32)


@pytest.mark.parametrize("M", [4, 100, 600])
def test_gemm_passes_nan_on_in_its_row_only(q8, M):
    qa, sa, qw, sw = operands(M, 256, 512, seed=2)
    sa[1, 2] = math.nan
    sa[2, 0] = math.inf
    y = q8.q8_gemm_fp8(qa.cuda(), sa.cuda(), qw.cuda(), sw.cuda(), out_dtype=torch.float32).cpu()
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    keep = [m for m in range(M) if m not in (1, 2)]
    check(y[keep], qa.view(torch.uint8)[keep].view(qa.dtype), sa[keep], qw, sw, torch.float32)


def test_gemm_empty_k(q8):
    y = torch.ones(3, 8, device="cuda")
    e = torch.empty(3, 0, device="cuda")
    q8.q8_gemm_fp8(e.to(torch.float8_e4m3fn), e, torch.empty(8, 0, device="cuda").to(torch.float8_e4m3fn),
                   torch.empty(1, 0, device="cuda"), out_dtype=torch.float32, out=y)
    assert (y == 0).all()


COUNTS = [
    [1], [0, 1, 0], [3, 0, 5, 1], [16, 17, 15, 0, 33], [130, 1, 0, 64, 257], [0, 0, 300], [40] * 9, [513, 2, 700],
    [1] * 40, [0] * 100 + [7] + [0] * 30, [1, 2, 3, 4, 5] * 40,
]


@pytest.mark.parametrize("i", range(len(COUNTS)))
@pytest.mark.parametrize("N,K", [(264, 400), (130, 1040)])
def test_grouped(q8, i, N, K):
    """Groups of any size, empty ones among them; rows before the first group and after the last are not written."""
    counts, dtype = COUNTS[i], DTYPES[i % 3]
    E, lead, tail = len(counts), i % 2 * 3, 2
    rows = lead + sum(counts) + tail
    qa, sa, qw, sw = operands(rows, N, K, seed=i, E=E)
    offsets = torch.tensor([lead] + [lead + sum(counts[:e + 1]) for e in range(E)], dtype=torch.int32)
    y = torch.full((rows, N), 5.0, dtype=dtype, device="cuda")
    q8.q8_gemm_fp8_grouped(qa.cuda(), sa.cuda(), qw.cuda(), sw.cuda(), offsets.cuda(), out_dtype=dtype, out=y)
    assert (y[:lead] == 5).all() and (y[rows - tail:] == 5).all()
    for e in range(E):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        if counts[e]:
            check(y[at], qa[at], sa[at], qw[e], sw[e], dtype)


@pytest.mark.parametrize("counts,N,K", [([900, 0, 1500], 1500, 272), ([300, 260, 0, 411], 900, 1040)])
def test_grouped_many_rows(q8, counts, N, K):
    """Whole tiles and ragged last ones of the kernels for many rows, in a group's middle and end."""
    rows, E = sum(counts), len(counts)
    qa, sa, qw, sw = operands(rows, N, K, seed=N, E=E)
    offsets = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32)
    y = q8.q8_gemm_fp8_grouped(qa.cuda(), sa.cuda(), qw.cuda(), sw.cuda(), offsets.cuda(), out_dtype=torch.float16)
    for e in range(E):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        if counts[e]:
            check(y[at], qa[at], sa[at], qw[e], sw[e], torch.float16)


def test_grouped_offsets_are_cut_to_the_rows(q8):
    qa, sa, qw, sw = operands(20, 136, 256, seed=4, E=3)
    offsets = torch.tensor([0, 8, 25, 90], dtype=torch.int32)
    y = torch.full((20, 136), 5.0, device="cuda")
    q8.q8_gemm_fp8_grouped(qa.cuda(), sa.cuda(), qw.cuda(), sw.cuda(), offsets.cuda(), out_dtype=torch.float32, out=y)
    check(y[:8], qa[:8], sa[:8], qw[0], sw[0], torch.float32)
    check(y[8:], qa[8:], sa[8:], qw[1], sw[1], torch.float32)


def test_on_another_stream(q8):
    qa, sa, qw, sw = operands(50, 256, 512, seed=6)
    dev = [t.cuda() for t in (qa, sa, qw, sw)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = torch.empty(50, 256, device="cuda")
    q8.q8_gemm_fp8(*dev, out_dtype=torch.float32, out=y, stream=side)
    side.synchronize()
    check(y, qa, sa, qw, sw, torch.float32)


# ------------------------------------------------------------------------------- sizes, refusals

def test_outputs_past_32_bit_offsets(q8):
    """More than 2^31 elements in x, the codes and y: the last rows are where they belong."""
    M, K = 131100, 16384
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = ref.tokens(3, K, seed=1).to(torch.bfloat16).cuda()
    q, s = q8.q8_quantize_fp8(x)
    wq, ws = ref.quantize(x[-3:].float().cpu())
    same_codes(q[-3:], wq)
    same_scales(s[-3:], ws)
    del x, q, s
    for M, N in ((65600, 32800), (40, (1 << 31) // 40 + 1000)):
        qa, sa, qw, sw = operands(64, 256, 16, seed=M)
        qa, sa = (t.repeat(ref.cdiv(M, 64), 1)[:M] for t in (qa.view(torch.uint8).cuda(), sa.cuda()))
        qw = qw.view(torch.uint8).cuda().repeat(ref.cdiv(N, 256), 1)[:N]
        sw = sw.cuda().repeat(ref.cdiv(N, 256), 1)[:ref.cdiv(N, 128)].contiguous()
        y = q8.q8_gemm_fp8(qa.view(torch.float8_e4m3fn), sa, qw.view(torch.float8_e4m3fn), sw, out_dtype=torch.bfloat16)
        rows, cols = slice(M - 40, M), slice((N - 300) // 128 * 128, N)
        part = [t.cpu() for t in (qa[rows], sa[rows], qw[cols], sw[cols.start // 128:])]
        check(y[rows, cols], part[0].view(torch.float8_e4m3fn), part[1], part[2].view(torch.float8_e4m3fn), part[3],
              torch.bfloat16)
        del qa, sa, qw, sw, y


def test_binding_refusals(q8):
    qa, sa, qw, sw = (t.cuda() for t in operands(8, 256, 256, seed=1))
    for change in (dict(sa=sa[:, :1]), dict(sa=sa.half()), dict(qa=qa[:, :240]), dict(sw=sw[:1]), dict(qa=qa.view(torch.uint8)),
                   dict(qw=qw.view(torch.uint8)), dict(out=torch.empty(8, 255, device="cuda", dtype=torch.bfloat16)),
                   dict(out=torch.empty(8, 256, device="cuda")), dict(out_dtype=torch.float64), dict(sw=sw.cpu())):
        with pytest.raises((TypeError, ValueError)):
            q8.q8_gemm_fp8(**{**dict(qa=qa, sa=sa, qw=qw, sw=sw), **change})
    with pytest.raises(ValueError):
        q8.q8_gemm_fp8_grouped(qa, sa, qw[None], sw[None], torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        q8.q8_gemm_fp8_grouped(qa, sa, qw[None], sw[None], torch.zeros(2, dtype=torch.int64, device="cuda"))
    x = torch.zeros((4, 256), device="cuda")
    with pytest.raises(ValueError):
        q8.q8_quantize_fp8(x, slots=torch.zeros((3, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        q8.q8_quantize_fp8(x, rows=5)
    with pytest.raises(ValueError):
        q8.q8_quantize_fp8(x[:1].expand(4, 256))
    with pytest.raises(q8.Q8Error):
        q8.q8_quantize_fp8(torch.zeros((4, 100), device="cuda"))
    with pytest.raises(ValueError):
        q8.q8_swiglu_quantize_fp8(torch.zeros((4, 33), device="cuda"))
    with pytest.raises(ValueError):
        q8.q8_moe_route(x, 2, score="relu")
    with pytest.raises(q8.Q8Error):
        q8.q8_moe_route(x, 257)
    with pytest.raises(ValueError):
        q8.q8_moe_combine(x[:, :128], torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros((1, 1), device="cuda"))


def test_nothing_to_do(q8):
    """No rows, no experts with rows, no answers: empty results, or zeros."""
    e = torch.empty((0, 256), device="cuda")
    q, s = q8.q8_quantize_fp8(e)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    qw, sw = q8.q8_quantize_weight_fp8(torch.randn((2, 128, 256), device="cuda"))
    assert q8.q8_gemm_fp8(q, s, qw[0], sw[0]).shape == (0, 128)
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert q8.q8_gemm_fp8_grouped(q, s, qw, sw, offsets).shape == (0, 128)
    q, s = q8.q8_quantize_fp8(torch.randn((5, 256), device="cuda"))
    y = torch.full((5, 128), 3.0, device="cuda")
    q8.q8_gemm_fp8_grouped(q, s, qw, sw, offsets, out_dtype=torch.float32, out=y)
    assert (y == 3).all()
    idx, w = q8.q8_moe_route(torch.empty((0, 8), device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    y = q8.q8_moe_combine(torch.empty((0, 64), device="cuda"), torch.full((3, 2), -1, dtype=torch.int32, device="cuda"),
                          torch.ones((3, 2), device="cuda"))
    assert y.shape == (3, 64) and (y == 0).all()
