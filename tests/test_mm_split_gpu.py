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


@pytest.mark.parametrize("M,N,K", [(64, 1536, 4096), (100, 1000, 4096), (33, 64, 4096)])
def test_nan_and_infinity_stay_in_their_rows(M, N, K):
    p = _problem(M, N, K, 6, aux=False)
    p["a"][0, 3] = 0x7F  # NaN, in the first CTA's part of K
    p["a"][M - 1, K - 5] = 0x7F  # and in the last one's
    out, z = _run(p, ops.ACT_GELU)
    for t in (out, z):
        assert torch.isnan(t[0]).all() and torch.isnan(t[-1]).all() and torch.isfinite(t[1:-1]).all()
    p["a"][0, 3] = p["a"][M - 1, K - 5] = 0
    p["bias"][5], p["bias"][6] = float("inf"), 1e30
    out, z = _run(p, ops.ACT_SILU)
    assert torch.isinf(out[:, 5]).all() and torch.isfinite(out[:, 6]).all() and torch.isfinite(out[:, 7:]).all()


@pytest.mark.parametrize("M,N,K", [(64, 1536, 4096), (100, 1000, 4096), (33, 64, 4096)])
def test_the_amax_ignores_nan_and_an_infinite_one_keeps_the_scale(M, N, K):
    p = _problem(M, N, K, 8, aux=False)
    p["a"][1, 7] = 0x7F
    keep = np.array([m for m in range(M) if m != 1])
    _, _, y, ty = _reference(p, ops.ACT_RELU, ops.AUX_ADD, keep)
    ring = ops.Ring(scale=3.0)
    out, _ = _run(p, ops.ACT_RELU, out_fmt=ops.E4M3, ring=ring)
    torch.cuda.synchronize()
    hist = ring.state()[0]
    assert abs(float(hist[0]) - np.abs(y).max()) <= ty.max()
    assert ((out[1] & 0x7F) == 0x7F).all() and not ((out[torch.from_numpy(keep).cuda()] & 0x7F) == 0x7F).any()
    p["bias"][9] = float("inf")
    out, _ = _run(p, ops.ACT_RELU, out_fmt=ops.E4M3, ring=ring)
    torch.cuda.synchronize()
    after = ring.state()
    assert float(after[0][1]) == float("inf") and after[2] == np.float32(448.0 / np.float32(hist[0]))
    assert (out[torch.from_numpy(keep).cuda()][:, 9] == 0x7E).all()  # saturated
