"""Router, plan and layer at the edges of their definition, against plain forms in 64 bits."""
import math

import pytest
import torch

from . import fp8_reference as ref
from .test_gpu_moe import check_route

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
