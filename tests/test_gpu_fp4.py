"""4-bit floating-point quantizers and products against plain forms: the quantizers bit for bit (they are defined in fp32
operations), the products against 64 bits within the bound of their fp32 sums and one output rounding."""
import math

import pytest
import torch

from . import fp4_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
BLOCKS = [16, 32]


@pytest.fixture(scope="module")
def q8():
    import int8_quantized_gemm_gb300 as q8
    yield q8
    torch.cuda.synchronize()
    assert q8.q8_device_error() == 0


def raw(t):
    return t.cpu().view(torch.uint8)


def same_rows(got, want, K, block, rows=None):
    """Codes, scales (with their padding) and row scales of a quantizer against ref.quantize's; rows that are whole only."""
    q, sf, s = got
    codes, wsf, ws = want
    rows = torch.arange(codes.shape[0]) if rows is None else rows
    assert torch.equal(q.cpu()[rows], ref.pack(codes)[rows])
    assert torch.equal(raw(sf)[rows], ref.pad(wsf, K, block)[rows])
    if block == 16:
        assert torch.equal(s.cpu()[rows], ws[rows])
    else:
        assert s is None


# ----------------------------------------------------------------------------------------- quantizers

@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (1, 256), (3, 288), (5, 1056), (64, 4096), (257, 544), (2, 16384), (3, 20000), (2, 33024)])
def test_quantize(q8, dtype, M, K, block):
    x = ref.tokens(M, K, seed=M + K).to(dtype)
    same_rows(q8.q8_quantize_fp4(x.cuda(), block=block), ref.quantize(x.float(), block), K, block)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_halfway(q8, dtype, block):
    """Values that lie halfway between two levels, both signs, and the levels themselves: to the even code."""
    grid = torch.arange(-24, 25) * 0.25                                 # steps of 1/4 from -6 to 6
    x = torch.zeros((4, 64))
    x[:, :49] = grid
    x[:, 16], x[:, 32], x[:, 48] = 6.0, -6.0, 6.0                       # each block's largest is 6
    x[:, 63] = 6.0
    x[1] *= 2.0 ** -7
    x[2] *= 2.0 ** 5
    x[3] *= -1.0
    x = x.to(dtype)
    want = ref.quantize(x.float(), block)
    same_rows(q8.q8_quantize_fp4(x.cuda(), block=block), want, 64, block)
    assert {int(c) & 7 for c in want[0][0].flatten()} == set(range(8))


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_extremes(q8, dtype, block):
    """Zero rows and blocks, subnormals, the type's largest value; infinities and NaN break their own row (block) only."""
    x = ref.tokens(9, 416, seed=3).to(dtype)
    x[0] = 0.0
    x[1, :] = torch.finfo(dtype).tiny
    x[2, 5] = torch.finfo(dtype).max
    x[3, 130] = math.inf
    x[4, 415] = -math.inf
    x[5, 128] = math.nan
    x[6, 0], x[6, 1] = math.nan, math.inf
    x[7] = -0.0
    x[8, 32:64] = torch.finfo(dtype).smallest_normal / 4
    got, want = q8.q8_quantize_fp4(x.cuda(), block=block), ref.quantize(x.float(), block)
    whole = torch.tensor([0, 1, 2, 7, 8])
    same_rows(got, want, 416, block, whole)
    q, sf, s = got
    # in 64 bits: fp32's largest value has the code 4 at 2^126, which is 2^128
    v = ref.values(ref.unpack(q.cpu()), raw(sf)[:, :416 // block].contiguous(), None if s is None else s.cpu(), block)
    assert torch.isfinite(v[whole]).all()
    if block == 16:
        assert torch.isnan(s[3:7]).all() and torch.isnan(v[3:7]).all()
    else:
        assert torch.equal(raw(sf), ref.pad(want[1], 416, block))
        assert torch.isnan(v[3, 128:160]).all() and torch.isfinite(v[3, :128]).all() and torch.isfinite(v[3, 160:]).all()


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_strided_rows(q8, dtype, block):
    base = ref.tokens(33, 512, seed=5).to(dtype).cuda()
    n = 16 // base.element_size()
    for x in (base[::2, 64:64 + 288], base[:, n:n + 96]):               # the second: rows on 16 bytes, not on 32
        same_rows(q8.q8_quantize_fp4(x, block=block), ref.quantize(x.float().cpu().contiguous(), block), x.shape[1], block)
    with pytest.raises(ValueError):
        q8.q8_quantize_fp4(base.t(), block=block)
    with pytest.raises(q8.Q8Error):
        q8.q8_quantize_fp4(base[:, 1:1 + 288], block=block)             # rows are not 16-byte aligned


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,k", [(1, 128, 1), (7, 416, 3), (65, 1024, 8), (2, 17408, 2)])
def test_quantize_to_slots(q8, dtype, M, K, k, block):
    """Rows go to their slots; slots outside the result are skipped and rows that nobody has stay."""
    x = ref.tokens(M, K, seed=M).to(dtype)
    g = torch.Generator().manual_seed(M)
    rows = M * k + 3
    slots = torch.randperm(rows, generator=g)[:M * k].to(torch.int32).view(M, k)
    slots[torch.rand((M, k), generator=g) < 0.2] = -1
    if M > 1:
        slots[0, 0] = rows                            # outside: skipped
    q = torch.full((rows, K // 2), 0x5A, dtype=torch.uint8)
    sf = torch.full((rows, ref.pitch(K, block)), 0x33, dtype=torch.uint8)
    s = torch.full((rows,), 7.0)
    codes, wsf, ws = ref.quantize(x.float(), block)
    got = q8.q8_quantize_fp4(x.cuda(), block=block, slots=slots.cuda(), rows=rows, q=q.cuda(), sf=sf.view(ref.SCALE[block]).cuda(),
                             s=s.cuda() if block == 16 else None)
    for m in range(M):
        for d in slots[m].tolist():
            if 0 <= d < rows:
                q[d], sf[d] = ref.pack(codes)[m], ref.pad(wsf, K, block)[m]
                if block == 16:
                    s[d] = ws[m]
    assert torch.equal(got[0].cpu(), q) and torch.equal(raw(got[1]), sf)
    assert got[2] is None if block == 32 else torch.equal(got[2].cpu(), s)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,I", [(1, 32), (3, 160), (130, 1056), (33, 2048), (2, 16896)])
def test_swiglu_quantize(q8, dtype, M, I, block):
    """The activation is off by less than 2^-20. Row scales within 2^-19, then; block scales within half a step of e4m3 (2^-4, or
    2^-10 of a subnormal) of the block's share, or the smallest power of two, of a maximum that much off; codes within half
    a step of the value they stand for, which is at most 1 between 4 and 6 and 1/4 below 2, or the levels' end."""
    h = ref.tokens(M, 2 * I, seed=I, outliers=False).to(dtype)
    q, sf, s = q8.q8_swiglu_quantize_fp4(h.cuda(), block=block)
    g, u = h[:, :I].double(), h[:, I:].double()
    x = g / (1.0 + torch.exp(-g)) * u
    b = x.view(M, I // block, block).abs().amax(2)
    near = 1 + 2.0 ** -18
    c = ref.scale_values(raw(sf)[:, :I // block].contiguous(), block)
    assert (raw(sf)[:, I // block:] == 0).all()
    if block == 16:
        a = b.amax(1).clamp_min(1e-30)
        s = s.cpu().double()
        assert ((s - a / 2688.0).abs() <= 2.0 ** -19 * a / 2688.0).all()
        share = b / (a / 448.0)[:, None]
        assert ((c - share).abs() <= torch.maximum(share * 2.0 ** -4, torch.tensor(2.0 ** -10).double()) * near).all()
        unit = c * s[:, None]
    else:
        assert (b <= 6.0 * c * near).all() and ((b * near > 3.0 * c) | (c == 2.0 ** -127)).all()
        unit = c
    codes = ref.unpack(q.cpu())
    v = ref.LEVELS.double()[codes.long()]
    unit = unit.repeat_interleave(block, 1)
    live = unit > 0
    t = x / unit.clamp_min(1e-300)
    size = t.abs()
    half = torch.where(size < 2, 0.25, torch.where(size < 4, 0.5, 1.0)).double()
    assert (((v - t).abs() <= half + size * 2.0 ** -18) | ((v.abs() == 6) & (size > 6)) | ~live).all()
    assert (codes[~live] & 7 == 0).all()


def test_swiglu_strided_and_extremes(q8):
    base = ref.tokens(9, 1024, seed=1, outliers=False).to(torch.bfloat16)
    base[1, 0], base[2, 3], base[3, 260] = math.nan, math.inf, -math.inf
    base[4, 0], base[4, 256] = -3e38, 1.0                            # silu of a very negative gate is -0
    h = base.cuda()[:, :512]
    q, sf, s = q8.q8_swiglu_quantize_fp4(h, block=16)
    assert torch.isnan(s[1:4]).all() and torch.isfinite(s[4:]).all() and torch.isfinite(s[0])
    assert int(q[4, 0]) & 7 == 0
    q, sf, s = q8.q8_swiglu_quantize_fp4(h, block=32)
    v = q8.q8_dequantize_fp4(q, sf, s, out_dtype=torch.float32)
    assert torch.isnan(v[1, :32]).all() and torch.isnan(v[2, :32]).all() and torch.isnan(v[3, :32]).all()
    assert torch.isfinite(v[1:4, 32:]).all() and torch.isfinite(v[4:]).all()


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,N,K", [(1, 1, 32), (1, 128, 256), (3, 130, 288), (2, 257, 1056)])
def test_quantize_weight(q8, dtype, E, N, K, block):
    w = (ref.tokens(E * N, K, seed=N) * 0.02).to(dtype).view(E, N, K)
    qw, sfw, sw = q8.q8_quantize_weight_fp4(w.cuda(), block=block)
    for e in range(E):
        codes, sf, s = ref.quantize(w[e].float(), block)
        assert torch.equal(qw[e].cpu(), ref.pack(codes))
        assert torch.equal(raw(sfw)[e], ref.tile(sf, K, block))
        assert sw is None if block == 32 else torch.equal(sw[e].cpu(), s)
        one = q8.q8_quantize_weight_fp4(w[e].cuda(), block=block)
        assert torch.equal(one[0], qw[e]) and torch.equal(raw(one[1]), raw(sfw)[e])


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize(q8, dtype, block):
    E, N, K = 2, 131, 352
    x = ref.tokens(E * N, K, seed=2)
    codes, sf, s = ref.quantize(x, block)
    f = ref.LEVELS[codes.long()] * ref.scale_values(sf, block).float().repeat_interleave(block, 1)
    want = (f if s is None else f * s[:, None]).to(dtype)
    got = q8.q8_dequantize_fp4(*q8.q8_quantize_fp4(x.cuda(), block=block), out_dtype=dtype)
    assert torch.equal(got.cpu(), want)
    got = q8.q8_dequantize_fp4(*q8.q8_quantize_weight_fp4(x.view(E, N, K).cuda(), block=block), out_dtype=dtype)
    assert torch.equal(got.cpu().view(E * N, K), want)


def test_dequantize_codes(q8):
    """Every pair of codes, alone and with a scale of each kind."""
    q = torch.arange(256, dtype=torch.uint8).view(2, 128).cuda()
    want = ref.LEVELS[ref.unpack(q.cpu()).long()]
    for dtype in (*DTYPES, torch.float8_e4m3fn):
        got = q8.q8_dequantize_fp4(q, out_dtype=dtype).cpu().float()
        assert torch.equal(got, want) and torch.equal(torch.signbit(got), torch.signbit(want))
    s = torch.tensor([3.0, -0.5]).cuda()
    assert torch.equal(q8.q8_dequantize_fp4(q, None, s, out_dtype=torch.float32).cpu(), want * s.cpu()[:, None])
    for block in BLOCKS:
        sf = torch.randint(0, 255, (2, 256 // block), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
        sf[0, :3] = torch.tensor([0, 1, 126])
        if block == 16:
            sf &= 0x7F
            sf[sf == 0x7F] = 0x7E
        got = q8.q8_dequantize_fp4(q, sf.view(ref.SCALE[block]).cuda(), out_dtype=torch.float32).cpu()
        assert torch.equal(got, want * ref.scale_values(sf, block).float().repeat_interleave(block, 1))


# ------------------------------------------------------------------------------------------- products

def device(op, block, weight=False):
    """Operands of a product on the GPU from ref.operand's."""
    _, q, rows, tiles, s = op
    return q.cuda(), (tiles if weight else rows).view(ref.SCALE[block]).cuda(), None if s is None else s.cuda()


def check(got, a, w, K, dtype):
    y, mag = ref.product(a, w)
    off = (got.cpu().double() - y).abs()
    tol = ref.product_tolerance(y, mag, K, dtype)
    assert (off <= tol).all(), f"off by up to {float((off / tol).max())} of the bound"
    return float((off / tol).max())


SIZES = [(1, 8, 32), (1, 128, 256), (3, 130, 288), (16, 264, 2048), (17, 1000, 544), (33, 257, 96), (64, 512, 1024),
         (65, 129, 4128), (100, 384, 320), (128, 256, 512), (129, 391, 800), (200, 264, 1088), (257, 520, 1312), (300, 1026, 64),
         (517, 2056, 2080), (1000, 700, 4096), (2600, 2599, 544), (2561, 4001, 96), (3333, 2600, 1312)]


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm(q8, M, N, K, block):
    a, w = ref.operand(M, K, block, seed=M), ref.operand(N, K, block, seed=N + 1, scale=0.02)
    for dtype in DTYPES:
        y = q8.q8_gemm_fp4(*device(a, block), *device(w, block, True), out_dtype=dtype)
        check(y, a[0], w[0], K, dtype)


@pytest.mark.parametrize("block", BLOCKS)
def test_gemm_scales_of_ones(q8, block):
    """Row scales may be left out, on either side, for either format."""
    M, N, K = 70, 200, 416
    a, w = ref.operand(M, K, block, seed=4), ref.operand(N, K, block, seed=5)
    (qa, sfa, sa), (qw, sfw, sw) = device(a, block), device(w, block, True)
    va, vw = a[0] if sa is None else a[0] / a[4].double()[:, None], w[0] if sw is None else w[0] / w[4].double()[:, None]
    check(q8.q8_gemm_fp4(qa, sfa, None, qw, sfw, None, out_dtype=torch.float32), va, vw, K, torch.float32)
    ones = torch.linspace(0.5, 2.0, M).cuda(), torch.linspace(-1.0, 1.0, N).cuda()
    got = q8.q8_gemm_fp4(qa, sfa, ones[0], qw, sfw, None, out_dtype=torch.float32)
    check(got, va * ones[0].cpu().double()[:, None], vw, K, torch.float32)
    got = q8.q8_gemm_fp4(qa, sfa, None, qw, sfw, ones[1], out_dtype=torch.float32)
    check(got, va, vw * ones[1].cpu().double()[:, None], K, torch.float32)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("M", [3, 40, 130, 600])
def test_gemm_broken_rows_stay_apart(q8, M, block):
    """A NaN in a token's or a weight's scales reaches its own row or column of y only; scales past K are not read."""
    N, K = 300, 288
    a, w = ref.operand(M, K, block, seed=6), ref.operand(N, K, block, seed=7)
    rows, tiles = a[2].clone(), w[3].clone()
    nan = 0x7F if block == 16 else 0xFF
    rows[:, K // block:] = nan
    sa = None if block == 32 else a[4].clone()
    if block == 16:
        sa[M // 2] = math.nan
    else:
        rows[M // 2, 1] = nan
    tiles[1, 1, 7, 2, 1] = nan                       # weight row 128 + 64 + 7, block 5
    q, sf, s = device(w, block, True)
    y = q8.q8_gemm_fp4(a[1].cuda(), rows.view(ref.SCALE[block]).cuda(), None if sa is None else sa.cuda(), q,
                       tiles.view(ref.SCALE[block]).cuda(), s, out_dtype=torch.float32).cpu()
    want = torch.zeros((M, N), dtype=torch.bool)
    want[M // 2], want[:, 199] = True, True
    assert torch.equal(torch.isnan(y), want)
    fine, cols = torch.arange(M) != M // 2, torch.arange(N) != 199
    check(y[fine][:, cols], a[0][fine], w[0][cols], K, torch.float32)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("M", [5, 100, 520])
def test_gemm_large_and_small_values(q8, M, block):
    """Rows of very different sizes: the products' scales neither overflow nor lose bits on the way."""
    N, K = 136, 1056
    x, v = ref.tokens(M, K, seed=8), ref.tokens(N, K, seed=9)
    x *= 2.0 ** torch.linspace(-60.0, 60.0, M).round()[:, None]
    v *= 2.0 ** torch.linspace(40.0, -40.0, N).round()[:, None]
    ops = []
    for t in (x, v):
        codes, sf, s = ref.quantize(t, block)
        ops.append((ref.values(codes, sf, s, block), ref.pack(codes), ref.pad(sf, K, block), ref.tile(sf, K, block), s))
    y = q8.q8_gemm_fp4(*device(ops[0], block), *device(ops[1], block, True), out_dtype=torch.float32)
    check(y, ops[0][0], ops[1][0], K, torch.float32)


def test_gemm_nothing_to_do(q8):
    for block in BLOCKS:
        a, w = ref.operand(4, 64, block, seed=1), ref.operand(8, 64, block, seed=2)
        (qa, sfa, sa), (qw, sfw, sw) = device(a, block), device(w, block, True)
        assert q8.q8_gemm_fp4(qa[:0], sfa[:0], None if sa is None else sa[:0], qw, sfw, sw).shape == (0, 8)
        y = q8.q8_gemm_fp4(qa, sfa, sa, qw[:0], sfw[:0], None if sw is None else sw[:0])
        assert y.shape == (4, 0)
        out = torch.full((4, 8), 3.0, dtype=torch.float16, device="cuda")
        q8.q8_gemm_fp4(qa[:, :0].contiguous(), sfa[:, :0].contiguous(), sa, qw[:, :0].contiguous(),
                       sfw[:, :0].contiguous(), sw, out_dtype=torch.float16, out=out)
        assert (out == 0).all()
        q, sf, s = q8.q8_quantize_fp4(torch.empty((0, 64), device="cuda"), block=block)
        assert q.shape == (0, 32) and sf.shape == (0, 256 // block)


def offsets_of(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32)


GROUPS = [
    ([3, 0, 5, 1], 130, 288),                    # a few rows; an expert without any
    ([0, 0, 1], 64, 32),
    ([17, 1, 0, 33, 2, 64], 264, 544),           # one tile and more of the smallest
    ([70, 130, 0, 1, 90], 257, 800),
    ([300, 1, 513, 0, 129], 392, 1312),          # CTA pairs; tiles that end in the next expert
    ([1000, 24], 640, 2080),
    ([3000, 1, 700, 0, 2000], 2050, 544),        # 256 x 256 tiles
    ([129, 2800, 2311], 2001, 800),
]


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("counts,N,K", GROUPS)
def test_grouped(q8, counts, N, K, block):
    """Every expert's rows with its own matrix, rows before the first and behind the last left as they were."""
    first, E = 5, len(counts)
    rows = first + sum(counts) + 7
    off = offsets_of(counts, first)
    a = ref.operand(rows, K, block, seed=N)
    ws = [ref.operand(N, K, block, seed=N + e + 1, scale=0.02) for e in range(E)]
    qw = torch.stack([w[1] for w in ws]).cuda()
    sfw = torch.stack([w[3] for w in ws]).view(ref.SCALE[block]).cuda()
    sw = torch.stack([w[4] for w in ws]).cuda() if block == 16 else None
    for dtype in DTYPES:
        out = torch.full((rows, N), -7.0, dtype=dtype, device="cuda")
        y = q8.q8_gemm_fp4_grouped(*device(a, block), qw, sfw, sw, off.cuda(), out_dtype=dtype, out=out)
        assert y is out and (y[:first] == -7).all() and (y[int(off[-1]):] == -7).all()
        for e in range(E):
            at = slice(int(off[e]), int(off[e + 1]))
            if counts[e]:
                check(y[at], a[0][at], ws[e][0], K, dtype)


@pytest.mark.parametrize("block", BLOCKS)
def test_grouped_offsets_of_any_value(q8, block):
    """Offsets past the rows are cut, falling ones end the call; nothing outside y is touched."""
    E, N, K, rows = 4, 72, 288, 50
    a = ref.operand(rows, K, block, seed=1)
    ws = [ref.operand(N, K, block, seed=e + 2) for e in range(E)]
    qw = torch.stack([w[1] for w in ws]).cuda()
    sfw = torch.stack([w[3] for w in ws]).view(ref.SCALE[block]).cuda()
    sw = torch.stack([w[4] for w in ws]).cuda() if block == 16 else None
    big = torch.full((rows + 200, N), 9.0, device="cuda")
    for off in ([0, 10, 60, 1 << 30, 1 << 30], [-5, 10, 20, 45, 50], [40, 10, 50, 0, 50], [50, 50, 50, 50, 50]):
        out = big[100:100 + rows]
        q8.q8_gemm_fp4_grouped(*device(a, block), qw, sfw, sw, torch.tensor(off, dtype=torch.int32).cuda(),
                               out_dtype=torch.float32, out=out)
        assert (big[:100] == 9).all() and (big[100 + rows:] == 9).all()
    y = q8.q8_gemm_fp4_grouped(*device(a, block), qw, sfw, sw, torch.tensor([0, 10, 60, 70, 90], dtype=torch.int32).cuda(),
                               out_dtype=torch.float32)
    check(y[:10], a[0][:10], ws[0][0], K, torch.float32)
    check(y[10:], a[0][10:], ws[1][0], K, torch.float32)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("M", [2, 96, 700])
def test_same_bits_again(q8, M, block):
    """The same call gives the same bits, on another stream, from a graph, and with another call's kernels beside it."""
    N, K = 520, 2080
    a, w = device(ref.operand(M, K, block, seed=1), block), device(ref.operand(N, K, block, seed=2), block, True)
    want = q8.q8_gemm_fp4(*a, *w)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        x, y = q8.q8_gemm_fp4(*a, *w, stream=other), q8.q8_gemm_fp4(*a, *w)
        torch.cuda.synchronize()
        assert torch.equal(x, want) and torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = q8.q8_gemm_fp4(*a, *w)
    for _ in range(3):
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, want)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("T", [1, 9, 300])
def test_layer_of_experts(q8, T, block):
    """The operators as a layer uses them, captured in a graph and replayed with other tokens, against 64 bits on the codes that the
    quantizers gave: both products within their bounds."""
    E, k, H, I = 6, 2, 288, 160
    g = torch.Generator().manual_seed(T)
    w13 = torch.randn((E, 2 * I, H), generator=g).cuda() * H ** -0.5
    w2 = torch.randn((E, H, I), generator=g).cuda() * I ** -0.5
    p13, p2 = q8.q8_quantize_weight_fp4(w13, block=block), q8.q8_quantize_weight_fp4(w2, block=block)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((T, E), generator=g).cuda()

    def layer():
        idx, weights = q8.q8_moe_route(logits, k)
        offsets, slots = q8.q8_moe_plan(idx, E)
        qa = q8.q8_quantize_fp4(x, block=block, slots=slots)
        h = q8.q8_gemm_fp4_grouped(*qa, *p13, offsets, out_dtype=torch.float32)
        qh = q8.q8_swiglu_quantize_fp4(h, block=block)
        z = q8.q8_gemm_fp4_grouped(*qh, *p2, offsets, out_dtype=torch.float32)
        return offsets, slots, weights, qa, h, qh, z, q8.q8_moe_combine(z, slots, weights)

    layer()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        offsets, slots, weights, qa, h, qh, z, y = layer()
    for turn in range(2):
        x.copy_(torch.randn((T, H), generator=g).to(torch.bfloat16))
        logits.copy_(torch.randn((T, E), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        off = offsets.tolist()
        codes, sf, s = ref.quantize(x.float().cpu(), block)
        for t in range(T):
            for d in slots[t].tolist():
                assert torch.equal(qa[0][d].cpu(), ref.pack(codes)[t])

        def value(q, sf, s):
            K = 2 * q.shape[-1]
            return ref.values(ref.unpack(q.cpu()), raw(sf)[:, :K // block].contiguous(), None if s is None else s.cpu(), block)
        va, vh = value(*qa), value(*qh)
        for e in range(E):
            at = slice(off[e], off[e + 1])
            if off[e] < off[e + 1]:
                check(h[at], va[at], q8.q8_dequantize_fp4(p13[0][e], p13[1][e], None if p13[2] is None else p13[2][e],
                                                          out_dtype=torch.float32).cpu().double(), H, torch.float32)
                check(z[at], vh[at], q8.q8_dequantize_fp4(p2[0][e], p2[1][e], None if p2[2] is None else p2[2][e],
                                                          out_dtype=torch.float32).cpu().double(), I, torch.float32)
        want = (weights.cpu().double()[:, :, None] * z.cpu().double()[slots.cpu().long()]).sum(1)
        size = (weights.cpu().double()[:, :, None] * z.cpu().double()[slots.cpu().long()].abs()).sum(1)
        assert ((y.cpu().double() - want).abs() <= 4 * 2.0 ** -24 * size + 1e-30).all()


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("M", [4, 24, 100, 3000])
def test_kernels_that_start_early_wait(q8, M, block):
    """Operands, scales, offsets and the result are rewritten right before and after each call on one stream, without a synchronisation
    between them: every kernel sees what the one before it wrote."""
    N, K, E = 1040, 1056, 3
    xs = [ref.tokens(M, K, seed=i).cuda() for i in range(3)]
    vs = [(ref.tokens(E * N, K, seed=10 + i) * 0.02).view(E, N, K).cuda() for i in range(3)]
    offs = [torch.tensor(o, dtype=torch.int32).cuda() for o in ([0, M // 2, M // 2, M], [0, 0, M // 4, M], [0, M, M, M])]
    want = []
    for x, v, off in zip(xs, vs, offs):
        a, w = q8.q8_quantize_fp4(x, block=block), q8.q8_quantize_weight_fp4(v, block=block)
        torch.cuda.synchronize()
        y = q8.q8_gemm_fp4_grouped(*a, *w, off, out_dtype=torch.float32)
        torch.cuda.synchronize()
        want.append((y, q8.q8_dequantize_fp4(a[0], a[1], a[2], out_dtype=torch.float32)))
        torch.cuda.synchronize()
    q, sf, s = q8.q8_quantize_fp4(xs[0], block=block)
    qw, sfw, sw = q8.q8_quantize_weight_fp4(vs[0], block=block)
    off, y, back = offs[0].clone(), torch.empty((M, N), device="cuda"), torch.empty((M, K), device="cuda")
    for turn in range(12):
        i = turn % 3
        off.copy_(offs[i])
        q8.q8_quantize_weight_fp4(vs[i], block=block, qw=qw, sfw=sfw, sw=sw)
        q8.q8_quantize_fp4(xs[i], block=block, q=q, sf=sf, s=s)
        q8.q8_gemm_fp4_grouped(q, sf, s, qw, sfw, sw, off, out_dtype=torch.float32, out=y)
        q8.q8_dequantize_fp4(q, sf, s, out_dtype=torch.float32, out=back)
        got = y.clone(), back.clone()
        q8.q8_gemm_fp4_grouped(q, sf, s, qw, sfw, sw, off, out_dtype=torch.float32, out=y)
        again = y.clone()
        y.fill_(-1.0)
        assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1]) and torch.equal(again, want[i][0])
