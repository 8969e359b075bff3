"""The product on both sides of the rule that picks the few-rows kernel."""

import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops
from gpu_helpers import require_gpu
from test_mm_act_gpu import _check, _problem

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# Long K in few rows (tiles, split and whole), the few-rows kernel's longest K, and 17 to 32
# rows on either side of each bound.
@pytest.mark.parametrize("M,N,K", [(1, 130, 16384), (8, 64, 8192), (8, 64, 8208), (3, 5000, 8192), (9, 200, 3328),
                                   (16, 200, 3344), (12, 1600, 4096), (16, 1537, 4112), (10, 8200, 4096),
                                   (24, 1536, 1024), (24, 1536, 1040), (20, 5120, 2560), (32, 7104, 2048),
                                   (32, 7120, 1024), (17, 4225, 1040)])
def test_either_kernel_within_the_bound(M, N, K):
    _check(_problem(M, N, K, M + K, rows=True), ops.ACT_SILU, ops.AUX_MUL, ops.E4M3)
    _check(_problem(M, N, K, M + K, bias=False), ops.ACT_GELU, ops.AUX_ADD, None)
