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


@pytest.mark.parametrize("out_fmt", [None, ops.E4M3])
@pytest.mark.parametrize("act", [ops.ACT_NONE, ops.ACT_RELU, ops.ACT_GELU, ops.ACT_SILU])
def test_equal_sums_give_equal_bits_in_every_kernel(act, out_fmt):
    """Operands of small whole numbers: their sums are exact in any order, so a row's result must
    not depend on how many rows are computed with it (few rows, a split K, whole tiles)."""
    N, K, M = 512, 4096, 4096
    g = torch.Generator().manual_seed(act)
    values = torch.tensor([-2.0, -1.0, 0.0, 1.0, 2.0]).to(torch.float8_e4m3fn).view(torch.uint8)
    a, b = (values[torch.randint(0, 5, (n, K), generator=g)].cuda() for n in (M, N))
    sa, sb = torch.rand(M, generator=g).cuda() * 0.02 + 0.02, torch.ones(1, device="cuda")
    bias, aux = torch.randn(N, generator=g).cuda(), torch.randn(M, N, generator=g).to(torch.bfloat16).cuda()

    def rows(m):
        ring = None if out_fmt is None else ops.Ring(scale=2.0)
        return ops.mm_act(a[:m], b, sa[:m], sb, act, bias=bias, aux=aux[:m], aux_op=ops.AUX_MUL, need_z=True,
                          out_fmt=out_fmt, out_ring=ring)

    out, z = rows(M)  # more tiles than there are pairs of CTAs: K stays whole
    for m in (1, 8, 16, 64, 200):
        o, zm = rows(m)
        assert torch.equal(zm, z[:m]) and torch.equal(o, out[:m]), m
    # Without K the sum is the bias, as with operands of zeros.
    ring, ring0 = (None if out_fmt is None else ops.Ring(scale=2.0) for _ in range(2))
    o, _ = ops.mm_act(a[:7, :16].contiguous() * 0, b[:, :16].contiguous() * 0, sb, sb, act, bias=bias, out_fmt=out_fmt,
                      out_ring=ring)
    e, f = (torch.empty(n, 0, dtype=torch.uint8, device="cuda") for n in (7, N))
    assert torch.equal(ops.mm_act(e, f, sb, sb, act, bias=bias, out_fmt=out_fmt, out_ring=ring0)[0], o)
