"""GPU: the calls around the grouped GEMMs where FP32, 31 bits, a cap or a second host thread can go wrong."""
import math
import threading

import pytest
import torch

from tests.test_gpu_moe import Layer, Layout, codes, scales
from tests.test_gpu_route import check_route, scores64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of FP32, relative


@pytest.fixture(scope="module")
def dgm():
    from moe_grouped_gemm_weight_b200 import build
    build.build()
    import moe_grouped_gemm_weight_b200 as dg
    dg.dg_set_num_sms(0)
    assert dg.dg_get_device_error() == 0
    return dg


@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (60, 5), (1020, 20)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_group_whose_sum_leaves_fp32_is_no_masked_group(dgm, E, groups, sigmoid, dtype):
    # The sum of two choice values at the lowest finite float is below every float, but the group has experts:
    # it stays behind the others, before masked ones.  Three experts of one group are ordinary, one group is masked.
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(7, E, generator=g).to(dtype)
    n = E // groups
    bias = torch.full((E,), torch.finfo(torch.float32).min)
    bias[n:2 * n] = -math.inf
    bias[2 * n:2 * n + 3] = 0.1
    bias[2 * n + 3:3 * n] = -math.inf
    check_route(dgm, logits, bias, k=8, groups=groups, keep=3, gtop=2, sigmoid=sigmoid, renorm=True, scale=1.0)
    check_route(dgm, logits, bias, k=8, groups=groups, keep=groups - 1, gtop=2, sigmoid=sigmoid)
