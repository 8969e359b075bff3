"""The order of every sum depends on sizes, type and device: the same values at other
addresses, which other loads serve, give the same bits."""

import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops
from gpu_helpers import require_gpu
from layer_helpers import DTYPES, at_offset

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _values(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * 0.37).to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(3000, 1536), (3000, 1537), (700, 256), (5000, 64), (1000, 2048), (400, 4096),
                                       (300, 12288), (100, 1024)])
def test_norm_backward_at_other_addresses(rows, cols, dtype):
    h, dy, dres = (_values(rows, cols, dtype, s) for s in (1, 2, 3))
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float().cuda()
    gamma = _values(1, cols, dtype, 4)[0] + 1
    want = None
    # Every tensor moved, one alone moved, and gamma alone: one of them is enough for the other loads.
    for o in ((0, 0, 0, 0), (1, 1, 1, 1), (3, 3, 3, 3), (0, 1, 0, 0), (0, 0, 0, 1)):
        dx, dg = ops.rmsnorm_backward(at_offset(dy, o[0]), at_offset(h, o[1]), rstd, at_offset(gamma, o[3]),
                                      at_offset(dres, o[2]))
        if want is None:
            want = dx, dg
        assert torch.equal(dx, want[0]) and torch.equal(dg, want[1]), o


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("rows,cols", [(1000, 1536), (200, 1537), (1200, 520), (3000, 4096)])
def test_act_backward_at_other_addresses(rows, cols, gate):
    dy, z, u = (_values(rows, cols, "bf16", s) for s in (5, 6, 7))
    want = None
    for o in (0, 1, 3):
        r = ops.act_backward(at_offset(dy, o), at_offset(z, o), ops.ACT_SILU, ops.E5M2, ops.Ring(),
                             u=at_offset(u, o) if gate else None, ring_u=ops.Ring() if gate else None, need_db=True)
        got = [t for t in r if t is not None]
        if want is None:
            want = got
        assert all(torch.equal(a, b) for a, b in zip(got, want)), o


@pytest.mark.parametrize("rows,cols", [(300, 1536), (50, 4096), (9, 8200), (700, 64)])
def test_norm_at_other_addresses(rows, cols):
    x, res = _values(rows, cols, "bf16", 8), _values(rows, cols, "bf16", 9)
    gamma = _values(1, cols, "bf16", 10)[0] + 1
    want = None
    for o in (0, 1, 3):
        r = ops.rmsnorm(at_offset(x, o), at_offset(gamma, o), at_offset(res, o), fmt=ops.E4M3, need_rstd=True,
                        need_y=True)
        if want is None:
            want = r
        assert all(torch.equal(a, b) for a, b in zip(r, want)), o
