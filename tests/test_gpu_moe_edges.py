"""Router, plan and layer at the edges of their definition, against plain forms in 64 bits."""
import math
import threading

import pytest
import torch

from . import fp8_reference as ref
from .test_gpu_moe import check_route, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8():
    import int8_quantized_gemm_gb300 as q8
    yield q8
    torch.cuda.synchronize()
    assert q8.q8_device_error() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group", [(256, 8, 4), (512, 4, 1), (96, 3, 2)])
def test_masking_bias_in_groups(q8, score, E, n_group, topk_group):
    """A bias of NaN or -inf takes its expert out of its group's score too, wherever it is among a lane's experts."""
    g = torch.Generator().manual_seed(E)
    bias = 0.1 * torch.randn(E, generator=g)
    off = torch.randperm(E, generator=g)[:E // 8]
    bias[off[::2]] = math.nan
    bias[off[1::2]] = -math.inf
    check_route(q8, torch.randn((600, E), generator=g), 8, bias, score=score, n_group=n_group, topk_group=topk_group)


def clock(call, calls=50):
    """Microseconds a call, the smallest of three rounds."""
    best = math.inf
    for _ in range(3):
        call()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        start.record()
        for _ in range(calls):
            call()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) * 1e3 / calls)
    return best


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_all_groups_kept(q8, score):
    """Where every group is kept there is nothing to decide between groups: the same choice as without them, and not
    every token again in 64 bits (which takes several times as long: 3 is between the two)."""
    g = torch.Generator().manual_seed(4)
    logits, bias = torch.randn((16384, 256), generator=g), 0.1 * torch.randn(256, generator=g)
    check_route(q8, logits[:300], 8, bias, score=score, n_group=8, topk_group=8)
    check_route(q8, logits[:300], 8, None, score=score, n_group=8, topk_group=8)
    l, b = logits.cuda(), bias.cuda()
    idx, w = q8.q8_moe_route(l, 8, score=score, bias=b)
    out = dict(idx=torch.empty_like(idx), weights=torch.empty_like(w))
    q8.q8_moe_route(l, 8, score=score, bias=b, n_group=8, topk_group=8, **out)
    assert torch.equal(out["idx"], idx)
    one = clock(lambda: q8.q8_moe_route(l, 8, score=score, bias=b, **out))
    all_kept = clock(lambda: q8.q8_moe_route(l, 8, score=score, bias=b, n_group=8, topk_group=8, **out))
    assert all_kept < 3.0 * one, (all_kept, one)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1e3, 1e4, 1e5, 1e7])
def test_groups_whose_biases_cancel(q8, score, size):
    """Two experts a group with biases of opposite sign: the group's score is small, the rounding of its terms is not."""
    g = torch.Generator().manual_seed(int(size))
    E = 16
    bias = size * (1.0 + torch.rand(E // 2, generator=g)).repeat_interleave(2)
    bias[1::2] *= -1.0
    check_route(q8, torch.randn((3000, E), generator=g), 4, bias, score=score, n_group=8, topk_group=4)


def test_group_scores_past_the_largest_fp32(q8):
    """Sums of two keys that only 64 bits tell apart; and whole groups that a very low bias puts last."""
    logits = torch.randn((40, 32), generator=torch.Generator().manual_seed(3))
    bias = torch.linspace(2.0e38, 3.3e38, 8).repeat_interleave(4)
    check_route(q8, logits, 4, bias, score="sigmoid", n_group=8, topk_group=3)
    check_route(q8, logits, 4, -bias, score="sigmoid", n_group=8, topk_group=3)
    bias = torch.zeros(32)
    bias[8:16] = torch.finfo(torch.float32).min
    check_route(q8, logits, 8, bias, score="softmax", n_group=8, topk_group=6)
    check_route(q8, logits, 8, bias, score="softmax", n_group=8, topk_group=7)


def test_sigmoid_of_very_low_logits(q8):
    """Scores down to fp32's subnormals. Of each: the exponential (2 steps, of 2^-149 where it is subnormal), a sum, a
    division, half a step each; renormalised, the same again of the sum, and the last division."""
    g = torch.Generator().manual_seed(6)
    logits = -86.0 - 8.0 * torch.rand((200, 8), generator=g)
    want_idx, want = ref.route(logits, 6, "sigmoid", renorm=False)
    idx, w = q8.q8_moe_route(logits.cuda(), 6, score="sigmoid", renorm=False)
    off = 4 * 2.0 ** -23 * want + 3 * 2.0 ** -149
    assert torch.equal(idx.cpu(), want_idx)
    assert ((w.cpu().double() - want).abs() <= off).all()
    idx, w = q8.q8_moe_route(logits.cuda(), 6, score="sigmoid")
    rel = off / want + (off.sum(1) / want.sum(1))[:, None] + 8 * 2.0 ** -24
    share = want / want.sum(1, keepdim=True)
    assert torch.equal(idx.cpu(), want_idx)
    assert ((w.cpu().double() - share).abs() <= share * rel * (1 + 2.0 ** -6)).all()


def test_layer_of_no_token(q8):
    """Every step of a routed layer with zero tokens: empty results, no error."""
    E, k, H, I = 8, 4, 256, 128
    w13 = q8.q8_quantize_weight_fp8(torch.randn((E, 2 * I, H), device="cuda"))
    w2 = q8.q8_quantize_weight_fp8(torch.randn((E, H, I), device="cuda"))
    x = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    y, idx, w = layer(q8, x, torch.empty((0, E), device="cuda"), None, w13, w2, k, E)
    assert y.shape == (0, H) and idx.shape == (0, k) and w.shape == (0, k)
    q, s = q8.q8_quantize_fp8(x, slots=torch.empty((0, k), dtype=torch.int32, device="cuda"), rows=3)
    assert q.shape == (3, H) and s.shape == (3, 2)


def test_plans_of_two_sizes_from_two_threads(q8):
    """The launch's shared memory limit is the same whatever the number of experts, so that one thread's call does not
    take the room from another's. The library is called without the binding, so that the calls overlap."""
    lib, wrong = q8.load(), []

    def work(E):
        idx = torch.randint(0, E, (8, 4), generator=torch.Generator().manual_seed(E)).to(torch.int32)
        want_o, want_s = ref.plan(idx, E)
        mine, stream = idx.cuda(), torch.cuda.Stream()
        offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        slots = torch.empty((8, 4), dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        args = (mine.data_ptr(), 8, 4, E, offsets.data_ptr(), slots.data_ptr(), stream.cuda_stream)
        status = [lib.q8_moe_plan(*args) for _ in range(20000)]
        stream.synchronize()
        if any(status) or not torch.equal(offsets.cpu(), want_o) or not torch.equal(slots.cpu(), want_s):
            wrong.append((E, sum(s != 0 for s in status)))

    threads = [threading.Thread(target=work, args=(E,)) for E in (380, 512, 400, 511)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
