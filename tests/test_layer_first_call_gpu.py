"""Each operator's first call in a process may be a captured one: nothing that it sets up on
the way is refused during a capture."""

import subprocess
import sys

import pytest

from conftest import ROOT
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
from fp8_delayed_scaling_02_b200 import ops
g = torch.Generator().manual_seed(0)
M = int(sys.argv[2])
x = torch.randn(M, 256, generator=g).to(torch.bfloat16).cuda()
w = (torch.randn(320, 256, generator=g) / 16).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
gamma, one = torch.ones(256, dtype=torch.bfloat16, device="cuda"), torch.ones(1, device="cuda")
rings = [ops.Ring() for _ in range(6)]

def call(r):
    n = ops.rmsnorm(x, gamma, x, fmt=ops.E4M3, ring=r[0], need_rstd=True)
    y, z = ops.mm_act(n.codes, w, n.sinv, one, ops.ACT_SILU, need_z=True, out_fmt=ops.E4M3, out_ring=r[1])
    a = ops.act_backward(z, z, ops.ACT_SILU, ops.E5M2, r[2], need_db=True)
    return [n.codes, y, a.dz, a.db, *ops.rmsnorm_backward(x, n.h, n.rstd, gamma)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call(rings[:3])
graph.replay()
want = call(rings[3:])
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("captured")
"""


@pytest.mark.parametrize("M", [4, 400])
def test_a_captured_call_may_be_the_first(M):
    require_gpu()
    r = subprocess.run([sys.executable, "-c", PROGRAM, ROOT, str(M)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


SPLIT_PROGRAM = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
from fp8_delayed_scaling_02_b200 import ops
g = torch.Generator().manual_seed(0)
a, b = ((torch.randn(n, 4096, generator=g) / 8).to(torch.float8_e4m3fn).view(torch.uint8).cuda() for n in (64, 512))
one = torch.ones(1, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = ops.mm_act(a, b, one, one, ops.ACT_GELU, need_z=True)
graph.replay()
want = ops.mm_act(a, b, one, one, ops.ACT_GELU, need_z=True)
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, want))
print("captured")
"""


def test_a_captured_product_with_a_split_k_may_be_the_first():
    require_gpu()
    r = subprocess.run([sys.executable, "-c", SPLIT_PROGRAM, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
