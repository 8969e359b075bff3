"""A product whose factor is a word of the ring it folds: the word as it was before the call."""

import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops
from gpu_helpers import require_gpu
from test_mm_act_gpu import _problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 4096, 512), (16, 256, 256), (64, 1536, 4096), (600, 1024, 512)])
@pytest.mark.parametrize("which", ["sinv_a", "sinv_b"])
def test_the_output_ring_may_hold_a_factor(M, N, K, which):
    require_gpu()
    p = _problem(M, N, K, 3)
    d = {k: p[k].cuda() for k in ("a", "b", "sinv_a", "sinv_b", "bias", "aux")}

    def ring():
        r = ops.Ring(scale=3.0)
        r.scale_inv.copy_(d[which])
        return r

    def call(r, factor):
        f = dict(sinv_a=d["sinv_a"], sinv_b=d["sinv_b"])
        f[which] = factor
        return ops.mm_act(d["a"], d["b"], f["sinv_a"], f["sinv_b"], ops.ACT_SILU, bias=d["bias"], aux=d["aux"],
                          need_z=True, out_fmt=ops.E4M3, out_ring=r)

    apart, within = ring(), ring()
    want, got = call(apart, d[which]), call(within, within.scale_inv)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(apart.buf, within.buf)
