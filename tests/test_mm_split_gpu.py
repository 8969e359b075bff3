"""The product whose tiles' K the CTAs of a cluster share: a CTA of a cluster that gives up,
and values that are not finite."""

import numpy as np
import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops
from gpu_helpers import require_gpu
from test_mm_act_gpu import _check, _problem, _reference, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    ops.debug_wait()  # defaults, whatever happened


@pytest.mark.parametrize("M,N,K", [(64, 1536, 4096), (100, 1000, 4096), (512, 1536, 4096), (65, 130, 16000)])
@pytest.mark.parametrize("local", [False, True])
def test_a_cta_that_gives_up_takes_its_cluster_with_it(M, N, K, local):
    """The first CTA of each cluster waits until its budget is spent and leaves no sums; the
    others finish theirs.  No CTA may join the parts, so that no amax but 0 reaches the ring."""
    p = _problem(M, N, K, 5)
    ring, amax = ops.Ring(scale=3.0), torch.full((1,), 7.0, device="cuda")
    before = ring.state()
    torch.cuda.synchronize()
    assert ops.device_error(clear=True)[0] == ops.FP8_OK
    ops.debug_wait(1_000_000, ops.SITE_SPLIT_ONE_CTA)
    try:
        _run(p, ops.ACT_SILU, ops.AUX_MUL, ops.E4M3, ring, out_amax=amax if local else None)
        torch.cuda.synchronize()
    finally:
        ops.debug_wait()
    rc, where = ops.device_error(clear=True)
    assert rc == ops.FP8_ERR_DEVICE_TIMEOUT and where == ops.SITE_EPILOGUE_TMEM_FULL, (rc, where)
    hist, idx, scale, _, scratch = ring.state()
    assert all(int(v) == 0 for v in scratch)
    assert torch.equal(hist, before[0]) and scale == 3.0  # an amax of 0 in a ring of zeros
    assert idx == (0 if local else 1)
    assert amax.item() == (0.0 if local else 7.0)
    _check(p, ops.ACT_SILU, ops.AUX_MUL, ops.E4M3)  # the next call is whole
