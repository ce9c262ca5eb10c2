"""Each of the kernels behind the 4-bit products, at sizes that reach it: scales left out, broken rows, values of very different size,
groups that end inside a tile, the same bits again, and operands that the kernel before has only just written. Every test looks
up which kernel its call launched."""
import ctypes
import math

import pytest
import torch

from . import fp4_reference as ref
from .test_gpu_fp4 import check, device, offsets_of, q8  # noqa: F401  (q8 is the fixture)

pytestmark = pytest.mark.gpu
BLOCKS = [16, 32]
SWAP, WIDE, PAIR = "gemm_fp4_swap_kernel", "gemm_fp4_wide_kernel", "gemm_fp4_pair_kernel"

# K is never whole spans of 256. Both forms of each kernel's stores: rows of y of whole 16-byte chunks, and others.
DENSE = [(SWAP, 3, 264, 1056), (SWAP, 200, 262, 1056), (WIDE, 517, 2056, 1056), (WIDE, 520, 2051, 1056), (PAIR, 1300, 1544, 800),
         (PAIR, 2600, 2571, 288)]
GROUPED = [(SWAP, [17, 1, 0, 33, 2, 64], 264, 544), (WIDE, [300, 1, 513, 0, 129], 1032, 1056), (WIDE, [129, 700, 411], 1030, 544),
           (PAIR, [300, 1, 513, 0, 129], 2056, 1312), (PAIR, [129, 700, 411], 2001, 1056)]


class KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("dims", ctypes.c_uint * 7), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def kernels_of(call):
    """Names of the kernels that a call launches: those of its captured graph."""
    cu = ctypes.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = call()
    handle, n, names = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0), []
    assert cu.cuGraphGetNodes(handle, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(handle, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        kind, p, name = ctypes.c_int(-1), KernelNode(), ctypes.c_char_p()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            got = (cu.cuKernelGetName(ctypes.byref(name), ctypes.c_void_p(p.kern)) if p.kern else
                   cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)))
            assert got == 0
            names.append(name.value.decode())
    del kept
    return names


def reaches(kernel, call):
    names = kernels_of(call)
    assert len(names) == 1 and kernel in names[0], names


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("kernel,M,N,K", DENSE)
def test_scales_of_ones(q8, kernel, M, N, K, block):
    """Row scales may be left out, on either side, for either format."""
    a, w = ref.operand(M, K, block, seed=4), ref.operand(N, K, block, seed=5)
    (qa, sfa, sa), (qw, sfw, sw) = device(a, block), device(w, block, True)
    va, vw = a[0] if sa is None else a[0] / a[4].double()[:, None], w[0] if sw is None else w[0] / w[4].double()[:, None]
    rows, cols = torch.linspace(0.5, 2.0, M), torch.linspace(-1.0, 1.0, N)
    reaches(kernel, lambda: q8.q8_gemm_fp4(qa, sfa, None, qw, sfw, None, out_dtype=torch.float32))
    for sa, xa in ((None, va), (rows, va * rows.double()[:, None])):
        for sw, xw in ((None, vw), (cols, vw * cols.double()[:, None])):
            got = q8.q8_gemm_fp4(qa, sfa, None if sa is None else sa.cuda(), qw, sfw, None if sw is None else sw.cuda(),
                                 out_dtype=torch.float32)
            check(got, xa, xw, K, torch.float32)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("kernel,M,N,K", DENSE)
def test_broken_rows_stay_apart(q8, kernel, M, N, K, block):
    """A NaN in a token's or a weight's scales reaches its own row or column of y only; tokens' scales past K are not read."""
    a, w = ref.operand(M, K, block, seed=6), ref.operand(N, K, block, seed=7)
    rows, tiles = a[2].clone(), w[3].clone()
    nan = 0x7F if block == 16 else 0xFF
    rows[:, K // block:] = nan
    broken = sorted({M // 2, M - 1})
    sa = None if block == 32 else a[4].clone()
    if block == 16:
        sa[broken] = math.nan
    else:
        rows[broken, 1] = nan
    cols = [199, N - 1]
    for n in cols:
        tiles[n // 128, 1, n % 32, n % 128 // 32, 1] = nan       # block 5
    q, sf, s = device(w, block, True)
    args = (a[1].cuda(), rows.view(ref.SCALE[block]).cuda(), None if sa is None else sa.cuda(), q,
            tiles.view(ref.SCALE[block]).cuda(), s)
    reaches(kernel, lambda: q8.q8_gemm_fp4(*args, out_dtype=torch.float32))
    y = q8.q8_gemm_fp4(*args, out_dtype=torch.float32).cpu()
    want = torch.zeros((M, N), dtype=torch.bool)
    want[broken], want[:, cols] = True, True
    assert torch.equal(torch.isnan(y), want)
    rest, kept = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    rest[broken], kept[cols] = False, False
    check(y[rest][:, kept], a[0][rest], w[0][kept], K, torch.float32)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("kernel,M,N,K", DENSE)
def test_large_and_small_values(q8, kernel, M, N, K, block):
    """Rows of very different sizes: the products' scales neither overflow nor lose bits on the way."""
    x, v = ref.tokens(M, K, seed=8), ref.tokens(N, K, seed=9)
    x *= 2.0 ** torch.linspace(-60.0, 60.0, M).round()[:, None]
    v *= 2.0 ** torch.linspace(40.0, -40.0, N).round()[:, None]
    ops = []
    for t in (x, v):
        codes, sf, s = ref.quantize(t, block)
        ops.append((ref.values(codes, sf, s, block), ref.pack(codes), ref.pad(sf, K, block), ref.tile(sf, K, block), s))
    a, w = device(ops[0], block), device(ops[1], block, True)
    reaches(kernel, lambda: q8.q8_gemm_fp4(*a, *w, out_dtype=torch.float32))
    check(q8.q8_gemm_fp4(*a, *w, out_dtype=torch.float32), ops[0][0], ops[1][0], K, torch.float32)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("kernel,M,N,K", DENSE)
def test_same_bits_again(q8, kernel, M, N, K, block):
    """The same call gives the same bits, on another stream, from a graph, and with another call's kernels beside it."""
    a, w = device(ref.operand(M, K, block, seed=1), block), device(ref.operand(N, K, block, seed=2), block, True)
    reaches(kernel, lambda: q8.q8_gemm_fp4(*a, *w))
    want = q8.q8_gemm_fp4(*a, *w)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(6):
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


def experts(counts, N, K, block, tail=7):
    """Tokens, the experts' matrices and the offsets; five rows lie before the first expert and `tail` behind the last."""
    off = offsets_of(counts, 5)
    rows = int(off[-1]) + tail
    ws = [ref.operand(N, K, block, seed=N + e + 1, scale=0.02) for e in range(len(counts))]
    qw = torch.stack([w[1] for w in ws]).cuda()
    sfw = torch.stack([w[3] for w in ws]).view(ref.SCALE[block]).cuda()
    sw = torch.stack([w[4] for w in ws]).cuda() if block == 16 else None
    return ref.operand(rows, K, block, seed=N), ws, (qw, sfw, sw), off


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("kernel,counts,N,K", GROUPED)
def test_tiles_that_end_in_the_next_expert(q8, kernel, counts, N, K, block):
    """Every expert's rows with its own matrix, whatever the rows beside them hold; rows of no expert as they were."""
    a, ws, w, off = experts(counts, N, K, block)
    rows, outside = a[2].clone(), torch.ones(a[2].shape[0], dtype=torch.bool)
    outside[5:int(off[-1])] = False
    rows[outside] = 0x7F if block == 16 else 0xFF                # scales of rows that belong to no expert: NaN
    sa = None if block == 32 else a[4].cuda()
    args = (a[1].cuda(), rows.view(ref.SCALE[block]).cuda(), sa, *w, off.cuda())
    reaches(kernel, lambda: q8.q8_gemm_fp4_grouped(*args, out_dtype=torch.float32))
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((len(rows), N), -7.0, dtype=dtype, device="cuda")
        q8.q8_gemm_fp4_grouped(*args, out_dtype=dtype, out=out)
        assert (out[outside.cuda()] == -7).all()
        for e, n in enumerate(counts):
            at = slice(int(off[e]), int(off[e + 1]))
            if n:
                check(out[at], a[0][at], ws[e][0], K, dtype)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("kernel,counts,N,K", GROUPED)
def test_operands_just_written(q8, kernel, counts, N, K, block):
    """Codes, both kinds of scales, row scales and offsets are rewritten by the kernels right before each call on one stream, by the
    quantizers (which let the product start early) and by others, without a synchronisation between them."""
    E, M = len(counts), sum(counts)
    turns = [counts, counts[::-1], counts[1:] + counts[:1]]
    offs = [offsets_of(c).cuda() for c in turns]
    xs = [ref.tokens(M, K, seed=i).cuda() for i in range(3)]
    vs = [(ref.tokens(E * N, K, seed=10 + i) * 0.02).view(E, N, K).cuda() for i in range(3)]
    want = []
    for x, v, off in zip(xs, vs, offs):
        a, w = q8.q8_quantize_fp4(x, block=block), q8.q8_quantize_weight_fp4(v, block=block)
        torch.cuda.synchronize()
        want.append(q8.q8_gemm_fp4_grouped(*a, *w, off, out_dtype=torch.float32))
        torch.cuda.synchronize()
    q, sf, s = q8.q8_quantize_fp4(xs[0], block=block)
    qw, sfw, sw = q8.q8_quantize_weight_fp4(vs[0], block=block)
    off, y = offs[0].clone(), torch.empty((M, N), device="cuda")
    reaches(kernel, lambda: q8.q8_gemm_fp4_grouped(q, sf, s, qw, sfw, sw, off, out_dtype=torch.float32))
    got = []
    for turn in range(12):
        i = turn % 3
        off.copy_(offs[i])
        first, last = (q8.q8_quantize_fp4, q8.q8_quantize_weight_fp4) if turn % 2 else (q8.q8_quantize_weight_fp4, q8.q8_quantize_fp4)
        for f in (first, last):
            if f is q8.q8_quantize_fp4:
                f(xs[i], block=block, q=q, sf=sf, s=s)
            else:
                f(vs[i], block=block, qw=qw, sfw=sfw, sw=sw)
        q8.q8_gemm_fp4_grouped(q, sf, s, qw, sfw, sw, off, out_dtype=torch.float32, out=y)
        got.append(y.clone())
        off.copy_(offs[(i + 1) % 3])
    torch.cuda.synchronize()
    for turn, y in enumerate(got):
        assert torch.equal(y, want[turn % 3])


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_results_read_as_soon_as_they_are_written(q8, dtype, block):
    """A chain of early-started kernels through the same buffers: product, gated quantizer, product, way back, tokens into slots."""
    M, H, I = 130, 544, 288
    g = torch.Generator().manual_seed(3)
    w1 = q8.q8_quantize_weight_fp4((torch.randn((2 * I, H), generator=g) * H ** -0.5).cuda(), block=block)
    w2 = q8.q8_quantize_weight_fp4((torch.randn((H, I), generator=g) * I ** -0.5).cuda(), block=block)
    xs = [torch.randn((M, H), generator=g).to(dtype).cuda() for _ in range(3)]
    slots = [torch.randperm(2 * M, generator=g).view(M, 2).int().cuda() for _ in range(3)]
    new = {}

    def steps(x, slot, wait, k):
        """k: the buffers, written again at each call."""
        wait()
        a = q8.q8_quantize_fp4(x, block=block, **k.get("a", new))
        wait()
        h = q8.q8_gemm_fp4(*a, *w1, out_dtype=dtype, **k.get("h", new))
        wait()
        b = q8.q8_swiglu_quantize_fp4(h, block=block, **k.get("b", new))
        wait()
        z = q8.q8_gemm_fp4(*b, *w2, out_dtype=dtype, **k.get("z", new))
        wait()
        c = q8.q8_quantize_fp4(z, block=block, slots=slot, **k.get("c", new))
        wait()
        back = q8.q8_dequantize_fp4(*c, out_dtype=torch.float32, **k.get("back", new))
        wait()
        return a, h, b, z, c, back

    want = [steps(x, s, torch.cuda.synchronize, {})[5] for x, s in zip(xs, slots)]
    a, h, b, z, c, back = steps(xs[0], slots[0], torch.cuda.synchronize, {})

    def parts(t):
        return dict(q=t[0], sf=t[1], **({} if t[2] is None else {"s": t[2]}))
    k = dict(a=parts(a), h=dict(out=h), b=parts(b), z=dict(out=z), c=parts(c), back=dict(out=back))
    slot, got = slots[0].clone(), []
    for turn in range(30):
        slot.copy_(slots[turn % 3])
        steps(xs[turn % 3], slot, lambda: None, k)
        got.append(back.clone())
    torch.cuda.synchronize()
    for turn, y in enumerate(got):
        assert torch.equal(y, want[turn % 3])
