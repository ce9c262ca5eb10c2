"""4-bit floating-point operators at the edges of what their documentation allows."""
import importlib.util
import os
import threading

import pytest
import torch

from . import fp4_reference as ref
from .test_gpu_fp8_edges import pool_stream

pytestmark = pytest.mark.gpu
BLOCKS = [16, 32]


@pytest.fixture(scope="module")
def q8():
    import int8_quantized_gemm_gb300 as q8
    yield q8
    torch.cuda.synchronize()
    assert q8.q8_device_error() == 0


def raw(t):
    return t.cpu().view(torch.uint8)


# ------------------------------------------------------------------------------------------ gates

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lo,hi,size", [(-20.0, -1.0, 1.0), (-60.0, -40.0, 1e4), (-87.0, -80.0, 3e30), (-103.0, -87.0, 3e34)])
def test_swiglu_of_closed_gates(q8, dtype, lo, hi, size):
    """Off by 2^-20 of the value and, where exp(-|g|) is not a normal number, by its two steps of 2^-149 times |g u| (as the float8
    operator, which shares the activation); then the scales' own rounding, and half a step of the codes."""
    M, I = 24, 288
    g = torch.Generator().manual_seed(int(-lo))
    gate = (lo + (hi - lo) * torch.rand((M, I), generator=g)).to(dtype)
    up = (torch.randn((M, I), generator=g).clamp(-1, 1) * size).to(dtype)
    q, sf, s = q8.q8_swiglu_quantize_fp4(torch.cat([gate, up], 1).cuda())
    gate, up = gate.double(), up.double()
    x = gate / (1.0 + torch.exp(-gate)) * up
    off = 2.0 ** -20 * x.abs() + 2.0 ** -148 * (gate * up).abs() * (gate < -87.3) + 2.0 ** -149
    a = x.abs().amax(1).clamp_min(1e-30)
    s = s.cpu().double()
    assert ((s * 2688.0 - a).abs() <= off.amax(1) + 2.0 ** -23 * a).all()
    unit = (ref.scale_values(raw(sf)[:, :I // 16].contiguous(), 16) * s[:, None]).repeat_interleave(16, 1)
    v = ref.LEVELS.double()[ref.unpack(q.cpu()).long()]
    live = unit > 0
    t, e = x / unit.clamp_min(1e-300), off / unit.clamp_min(1e-300)
    half = torch.where(t.abs() < 2, 0.25, torch.where(t.abs() < 4, 0.5, 1.0)).double()
    assert (((v - t).abs() <= half + e + t.abs() * 2.0 ** -20) | ((v.abs() == 6) & (t.abs() > 6)) | ~live).all()


# ------------------------------------------------------------------------------------------ sizes

@pytest.mark.parametrize("N", [33000, 33001])
def test_output_past_32_bit_offsets(q8, N):
    """More than 2^31 values of y: whole rows of 16-byte chunks (stores by TMA), and rows that are not."""
    M, K, block = 65600, 64, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, K), generator=g, device="cuda")
    w = torch.randn((N, K), generator=g, device="cuda")
    a, b = q8.q8_quantize_fp4(x, block=block), q8.q8_quantize_weight_fp4(w, block=block)
    y = q8.q8_gemm_fp4(*a, *b, out_dtype=torch.float16)
    rows = torch.tensor([0, 1, 255, 256, 32767, 65000, M - 130, M - 2, M - 1], device="cuda")
    va = q8.q8_dequantize_fp4(*a, out_dtype=torch.float32)[rows].double().cpu()
    vw = q8.q8_dequantize_fp4(*b, out_dtype=torch.float32).double().cpu()
    want, mag = ref.product(va, vw)
    assert ((y[rows].cpu().double() - want).abs() <= ref.product_tolerance(want, mag, K, torch.float16)).all()


def test_quantizer_past_32_bit_offsets(q8):
    """More than 2^31 values in, and codes and values back past that many bytes."""
    M, K = 131100, 16416
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 65535, 131000, M - 1], device="cuda")
    x[at] = ref.tokens(5, K, seed=1).to(torch.bfloat16).cuda()
    q, sf, s = q8.q8_quantize_fp4(x)
    codes, wsf, ws = ref.quantize(x[at].float().cpu(), 16)
    assert torch.equal(q[at].cpu(), ref.pack(codes)) and torch.equal(raw(sf[at]), ref.pad(wsf, K, 16)) and torch.equal(s[at].cpu(), ws)
    assert int(q[131050:131060].max()) == 0
    del x
    v = q8.q8_dequantize_fp4(q, sf, s, out_dtype=torch.bfloat16)
    want = (ref.LEVELS[codes.long()] * ref.scale_values(wsf, 16).float().repeat_interleave(16, 1) * ws[:, None]).to(torch.bfloat16)
    assert torch.equal(v[at].cpu(), want)


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("E,rows", [(512, 700), (512, 9000), (300, 40), (1, 77)])
def test_many_experts(q8, block, E, rows):
    N, K = 40, 96
    g = torch.Generator().manual_seed(E + rows)
    owner = torch.randint(0, E, (rows,), generator=g).sort().values
    offsets = torch.searchsorted(owner, torch.arange(E + 1)).to(torch.int32)
    x, w = torch.randn((rows, K), generator=g), torch.randn((E * N, K), generator=g)
    a = q8.q8_quantize_fp4(x.cuda(), block=block)
    b = q8.q8_quantize_weight_fp4(w.view(E, N, K).cuda(), block=block)
    y = q8.q8_gemm_fp4_grouped(*a, *b, offsets.cuda(), out_dtype=torch.float32).cpu().double()
    va = q8.q8_dequantize_fp4(*a, out_dtype=torch.float32).cpu().double()
    vw = q8.q8_dequantize_fp4(*b, out_dtype=torch.float32).cpu().double()[owner]
    want, mag = (vw @ va[:, :, None])[:, :, 0], (vw.abs() @ va.abs()[:, :, None])[:, :, 0]
    assert ((y - want).abs() <= ref.product_tolerance(want, mag, K, torch.float32)).all()


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("rows,N,K", [(16, 128, 256), (600, 520, 544), (4000, 2056, 1056)])
def test_overlapping_ranges_end(q8, block, rows, N, K):
    """Offsets that fall: the call ends, no more than disjoint ranges' work is done, and a disjoint call after it is right."""
    E = 40 if rows == 16 else 4
    g = torch.Generator().manual_seed(rows)
    a = q8.q8_quantize_fp4(torch.randn((rows, K), generator=g).cuda(), block=block)
    b = q8.q8_quantize_weight_fp4(torch.randn((E, N, K), generator=g).cuda(), block=block)
    y = torch.full((rows, N), 5.0, device="cuda")
    if E == 40:
        offsets = torch.tensor([0, 8] * 20 + [16], dtype=torch.int32)      # the 21st range of rows is not computed
        q8.q8_gemm_fp4_grouped(*a, *b, offsets.cuda(), out_dtype=torch.float32, out=y)
        assert (y[8:] == 5).all() and (y[:8] != 5).any()
        return
    q8.q8_gemm_fp4_grouped(*a, *b, torch.tensor([0, rows, 0, rows, rows // 2], dtype=torch.int32).cuda(), out_dtype=torch.float32, out=y)
    offsets = [0, rows // 3, rows // 3, rows - 7, rows]
    q8.q8_gemm_fp4_grouped(*a, *b, torch.tensor(offsets, dtype=torch.int32).cuda(), out_dtype=torch.float32, out=y)
    va = q8.q8_dequantize_fp4(*a, out_dtype=torch.float32).cpu().double()
    for e in (0, 2, 3):
        at = slice(offsets[e], offsets[e + 1])
        vw = q8.q8_dequantize_fp4(*(None if t is None else t[e] for t in b), out_dtype=torch.float32).cpu().double()
        want, mag = ref.product(va[at], vw)
        assert ((y[at].cpu().double() - want).abs() <= ref.product_tolerance(want, mag, K, torch.float32)).all()


@pytest.mark.parametrize("block", BLOCKS)
def test_views_of_larger_buffers(q8, block):
    """Operands and results that begin inside other tensors, on 16 bytes but on no more; what lies around them stays."""
    M, N, K = 37, 72, 288
    x = ref.tokens(M, K, seed=1)
    want = q8.q8_quantize_fp4(x.cuda(), block=block)
    P = ref.pitch(K, block)
    room = torch.full((4096 + M * K,), 0x77, dtype=torch.uint8, device="cuda")
    q, sf = room[16:16 + M * K // 2].view(M, K // 2), room[8208:8208 + M * P].view(ref.SCALE[block]).view(M, P)
    keep = room.clone()
    q8.q8_quantize_fp4(x.cuda(), block=block, q=q[:], sf=sf, s=want[2])
    assert torch.equal(q, want[0]) and torch.equal(raw(sf), raw(want[1]))
    room[16:16 + M * K // 2], room[8208:8208 + M * P] = 0x77, 0x77
    assert torch.equal(room, keep)
    w = q8.q8_quantize_weight_fp4(ref.tokens(2 * N, K, seed=2).view(2, N, K).cuda(), block=block)
    y = q8.q8_gemm_fp4(*want, *(None if t is None else t[1] for t in w), out_dtype=torch.float32)      # the second of two matrices
    big = torch.full((M + 2, N), 4.0, device="cuda")
    q8.q8_gemm_fp4(*want, *(None if t is None else t[1] for t in w), out_dtype=torch.float32, out=big[1:-1])
    assert torch.equal(big[1:-1], y) and (big[0] == 4).all() and (big[-1] == 4).all()
    back = torch.full((M * K + 8,), 3.0, dtype=torch.bfloat16, device="cuda")
    q8.q8_dequantize_fp4(*want, out=back[8:].view(M, K))
    assert torch.equal(back[8:].view(M, K), q8.q8_dequantize_fp4(*want)) and (back[:8] == 3).all()
    one = q8.q8_dequantize_fp4(want[0], out_dtype=torch.float8_e4m3fn)
    byte = torch.zeros(M * K + 16, dtype=torch.uint8, device="cuda")
    q8.q8_dequantize_fp4(want[0], out_dtype=torch.float8_e4m3fn, out=byte[16:].view(torch.float8_e4m3fn).view(M, K))
    assert torch.equal(byte[16:].view(M, K), one.view(torch.uint8)) and (byte[:16] == 0).all()


# ---------------------------------------------------------------------------------- streams, threads

def test_results_are_allocated_for_the_stream_that_writes_them(q8):
    def calls(stream):
        x, w = torch.randn((40, 256), device="cuda"), torch.randn((4, 256, 256), device="cuda")
        offsets = torch.tensor([0, 10, 10, 30, 40], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        kept = [x, w, offsets]
        a, b = q8.q8_quantize_fp4(x, stream=stream), q8.q8_quantize_weight_fp4(w, stream=stream)
        h = q8.q8_gemm_fp4_grouped(*a, *b, offsets, stream=stream)
        y = q8.q8_gemm_fp4(*a, *(t[0] for t in b), stream=stream)
        c = q8.q8_swiglu_quantize_fp4(h, stream=stream)
        v = q8.q8_dequantize_fp4(*a, stream=stream), q8.q8_dequantize_fp4(a[0], stream=stream)
        torch.cuda.synchronize()
        return kept, (*a, *b, h, y, *c, *v)

    side = torch.cuda.Stream()
    kept, results = calls(side)
    assert {pool_stream(t) for t in results} == {side.cuda_stream}
    assert side.cuda_stream not in {pool_stream(t) for t in kept}
    kept, results = calls(None)
    assert {pool_stream(t) for t in results} == {pool_stream(kept[0])} != {side.cuda_stream}


def test_several_threads(q8):
    """Threads with streams of their own, each with its own sizes (and so kernels), give what a thread alone gives."""
    sizes = [(3, 520, 544, 16), (29, 264, 1056, 32), (120, 700, 320, 16), (3000, 2600, 288, 32)]
    work = []
    for i, (M, N, K, block) in enumerate(sizes):
        x, w = ref.tokens(M, K, seed=i).cuda(), ref.tokens(N, K, seed=10 + i).cuda()
        a, b = q8.q8_quantize_fp4(x, block=block), q8.q8_quantize_weight_fp4(w, block=block)
        work.append((x, b, block, a[0], q8.q8_gemm_fp4(*a, *b)))
    torch.cuda.synchronize()
    wrong = []

    def go(x, b, block, codes, y):
        stream = torch.cuda.Stream()
        for _ in range(20):
            a = q8.q8_quantize_fp4(x, block=block, stream=stream)
            got = q8.q8_gemm_fp4(*a, *b, stream=stream)
            stream.synchronize()
            if not (torch.equal(a[0], codes) and torch.equal(got, y)):
                wrong.append(x.shape)

    threads = [threading.Thread(target=go, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_graphs_replayed_at_once(q8):
    """Two captured products on two streams share nothing."""
    pairs = []
    for i, (M, N, K) in enumerate([(20, 1040, 2080), (300, 520, 1056)]):
        a = q8.q8_quantize_fp4(ref.tokens(M, K, seed=i).cuda())
        b = q8.q8_quantize_weight_fp4(ref.tokens(N, K, seed=5 + i).cuda())
        want = q8.q8_gemm_fp4(*a, *b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = q8.q8_gemm_fp4(*a, *b)
        pairs.append((graph, torch.cuda.Stream(), y, want, a, b))
    for _ in range(10):
        for graph, stream, y, *_ in pairs:
            y.zero_()
        torch.cuda.synchronize()
        for graph, stream, y, *_ in pairs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for _, _, y, want, *_ in pairs)


def test_graph_with_branches(q8):
    """A capture that forks to another stream after the quantizer and joins again: replayed with other tokens."""
    w = [q8.q8_quantize_weight_fp4(ref.tokens(520, 1056, seed=i).cuda()) for i in range(2)]
    x = ref.tokens(40, 1056, seed=3).cuda()
    side = torch.cuda.Stream()

    def work():
        a = q8.q8_quantize_fp4(x)
        fork, join = torch.cuda.Event(), torch.cuda.Event()
        fork.record()
        with torch.cuda.stream(side):
            side.wait_event(fork)
            y1 = q8.q8_gemm_fp4(*a, *w[1], out_dtype=torch.float32)
            b = q8.q8_quantize_fp4(y1[:, :512])
            join.record()
        y0 = q8.q8_gemm_fp4(*a, *w[0], out_dtype=torch.float32)
        torch.cuda.current_stream().wait_event(join)
        return q8.q8_quantize_fp4(y0[:, :512] + y1[:, :512]), b, y0, y1

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both, b, y0, y1 = work()
    for turn in range(4):
        x.copy_(ref.tokens(40, 1056, seed=10 + turn))
        graph.replay()
        torch.cuda.synchronize()
        a = q8.q8_quantize_fp4(x)
        want = [q8.q8_gemm_fp4(*a, *v, out_dtype=torch.float32) for v in w]
        assert torch.equal(y0, want[0]) and torch.equal(y1, want[1])
        for got, t in ((both, want[0][:, :512] + want[1][:, :512]), (b, want[1][:, :512])):
            assert all(torch.equal(g.view(torch.uint8), v.view(torch.uint8)) for g, v in zip(got, q8.q8_quantize_fp4(t)))


# ------------------------------------------------------------------------------------------ the two ways a call is made

@pytest.mark.parametrize("block", BLOCKS)
def test_the_binding_makes_the_same_calls_itself(q8, block, monkeypatch):
    """Results of the compiled calls against those of the binding's own: types, shapes, bits, and the stream that is current."""
    assert q8._calls is not None
    x = ref.tokens(70, 544, seed=1).to(torch.bfloat16).cuda()
    slots = torch.randperm(140, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(70, 2).cuda()
    w = q8.q8_quantize_weight_fp4(ref.tokens(2 * 264, 544, seed=2).view(2, 264, 544).cuda(), block=block)
    off = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    h = ref.tokens(9, 320, seed=3).cuda()

    def calls():
        a = q8.q8_quantize_fp4(x, block=block)
        yield from a
        yield from q8.q8_quantize_fp4(x[::2, 32:320], block=block)
        yield from q8.q8_quantize_fp4(x, block=block, slots=slots)
        yield from q8.q8_quantize_fp4(x[:0], block=block)
        yield from q8.q8_swiglu_quantize_fp4(h, block=block)
        for t in (torch.float8_e4m3fn, torch.float16):
            yield q8.q8_dequantize_fp4(a[0], out_dtype=t)
        for t in (torch.float32, torch.bfloat16):
            yield q8.q8_gemm_fp4(*a, *(None if t is None else t[0] for t in w), out_dtype=t)
            yield q8.q8_gemm_fp4(*a[:2], None, *(None if t is None else t[1] for t in w[:2]), None, out_dtype=t)
            yield q8.q8_gemm_fp4_grouped(*a, *w, off, out_dtype=t)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        compiled = list(calls())
        side.synchronize()
    assert {pool_stream(t) for t in compiled if t is not None and t.numel()} == {side.cuda_stream}
    monkeypatch.setattr(q8, "_calls", None)
    own = list(calls())
    torch.cuda.synchronize()
    assert len(own) == len(compiled)
    for a, b in zip(compiled, own):
        if a is None or b is None:
            assert a is b
            continue
        assert (a.dtype, a.shape, a.device, a.stride()) == (b.dtype, b.shape, b.device, b.stride())
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------------------------------ refusals

def test_operands_that_do_not_fit_one_another(q8):
    a = q8.q8_quantize_fp4(torch.zeros((4, 256), device="cuda"))
    m = q8.q8_quantize_fp4(torch.zeros((4, 256), device="cuda"), block=32)
    w = q8.q8_quantize_weight_fp4(torch.zeros((130, 256), device="cuda"))
    e = q8.q8_quantize_weight_fp4(torch.zeros((2, 130, 256), device="cuda"))
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    cases = [
        lambda: q8.q8_gemm_fp4(*m, *w),                                         # blocks of 32 with blocks of 16
        lambda: q8.q8_gemm_fp4(a[0], a[1][:, :8], a[2], *w),                    # scales of too few K
        lambda: q8.q8_gemm_fp4(a[0], a[1], a[2][:3], *w),
        lambda: q8.q8_gemm_fp4(*a, w[0], w[1][:1], w[2]),                       # tiles of too few rows
        lambda: q8.q8_gemm_fp4(*a, w[0], a[1], w[2]),                           # rows of scales for tiles
        lambda: q8.q8_gemm_fp4(*a, *e),
        lambda: q8.q8_gemm_fp4(a[0][:, :64], a[1], a[2], *w),
        lambda: q8.q8_gemm_fp4(*a, *w, out_dtype=torch.int8),
        lambda: q8.q8_gemm_fp4(*a, *w, out=torch.empty((4, 131), dtype=torch.bfloat16, device="cuda")),
        lambda: q8.q8_gemm_fp4_grouped(*a, *e, off[:2]),
        lambda: q8.q8_gemm_fp4_grouped(*a, *e, off.long()),
        lambda: q8.q8_gemm_fp4_grouped(*a, *w, off),
        lambda: q8.q8_dequantize_fp4(a[0], a[1][:, :8].contiguous()),
        lambda: q8.q8_dequantize_fp4(a[0], a[1], a[2], out_dtype=torch.float8_e4m3fn),
        lambda: q8.q8_dequantize_fp4(e[0], a[1]),
        lambda: q8.q8_dequantize_fp4(a[0].t()),
        lambda: q8.q8_quantize_fp4(torch.zeros((4, 48), device="cuda")),
        lambda: q8.q8_quantize_fp4(torch.zeros((4, 64), device="cuda"), block=64),
        lambda: q8.q8_quantize_fp4(torch.zeros((4, 64), device="cuda"), block=32, s=torch.zeros(4, device="cuda")),
        lambda: q8.q8_quantize_fp4(torch.zeros((4, 64), device="cuda"), rows=5),
        lambda: q8.q8_swiglu_quantize_fp4(torch.zeros((4, 63), device="cuda")),
        lambda: q8.q8_quantize_weight_fp4(torch.zeros((4, 4, 4, 32), device="cuda")),
    ]
    for i, call in enumerate(cases):
        with pytest.raises((ValueError, TypeError, q8.Q8Error)):
            call()
            pytest.fail(f"case {i} was taken")


@pytest.mark.parametrize("fmt", ["fp4-16", "fp4-32"])
def test_example_of_a_layer(q8, fmt):
    """examples/moe_layer.py runs with 4-bit weights, with sizes that are no multiple of a tile."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main(["--experts", "12", "--top-k", "3", "--hidden", "544", "--inter", "288", "--tokens", "1,7,130", "--format", fmt])
