"""Codes on a ring and the factor that goes with them: the ring's word, until the next call."""

import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops
from gpu_helpers import OF, require_gpu
from layer_helpers import f64

pytestmark = pytest.mark.gpu


def test_two_forwards_on_one_ring_before_the_first_one_s_backward():
    require_gpu()
    g = torch.Generator().manual_seed(0)
    x = torch.randn(40, 256, generator=g).to(torch.bfloat16).cuda()
    gamma = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    ring = ops.Ring(scale=8.0)
    first = ops.rmsnorm(x, gamma, fmt=ops.E4M3, ring=ring, need_y=True)
    kept = first.sinv.clone()
    ops.rmsnorm(x * 3, gamma, fmt=ops.E4M3, ring=ring)  # on the scale that the first call published
    assert kept.item() == 0.125 and first.sinv is ring.scale_inv and first.sinv.item() != 0.125
    y = f64(first.y)
    got = OF.decode(first.codes.cpu().numpy(), OF.E4M3) * kept.item()
    # The code's rounding, its subnormal step, and y's own rounding to bf16.
    assert (abs(got - y) <= (2.0 ** -4 + 2.0 ** -7) * abs(y) + 2.0 ** -10 / 8).all()
