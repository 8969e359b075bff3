"""GPU parity of the activation's gradient with its FP8 casts and bias gradients against the oracle."""

import numpy as np
import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops
from gpu_helpers import require_gpu
from layer_helpers import DTYPES, U, assert_codes, assert_folded, assert_within, at_offset, f64
from oracle import act as OA

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (33, 1537), (40, 65), (257, 1024), (1000, 130), (2, 8200), (1, 4096)]
ACTS = [ops.ACT_NONE, ops.ACT_RELU, ops.ACT_GELU, ops.ACT_SILU]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _inputs(rows, cols, dtype, seed, gate):
    g = torch.Generator().manual_seed(seed)
    dy = (torch.randn(rows, cols, generator=g) * 1e-2).to(DTYPES[dtype])
    z = (torch.randn(rows, cols, generator=g) * 2).to(torch.bfloat16)
    u = torch.randn(rows, cols, generator=g).to(torch.bfloat16) if gate else None
    return dy, z, u


def _sums(got, ref, terms, err, what):
    # A sum of R terms in any order rounds at most R - 1 times; each term has its own error.
    tol = (terms.shape[0] + 1) * U * np.sum(np.abs(terms), axis=0) + np.sum(err, axis=0) + 2.0 ** -149
    assert_within(f64(got), ref, tol, what)


def _check(dy, z, u, act, fmt, db, offset=0, scale=30.0):
    ring, ring_u = ops.Ring(scale=scale), ops.Ring(scale=scale / 2) if u is not None else None
    before, before_u = ring.state(), ring_u.state() if u is not None else None
    r = ops.act_backward(at_offset(dy, offset), None if z is None else at_offset(z, offset), act, fmt, ring,
                         None if u is None else at_offset(u, offset), ring_u, need_db=db)
    torch.cuda.synchronize()
    d, zz = f64(dy), np.zeros(dy.shape) if z is None else f64(z)
    dz, du = OA.backward(d, zz, act, None if u is None else f64(u))
    lead = np.abs(d) * (1.0 if u is None else np.abs(f64(u)))
    # The slope's own error, and one rounding each of dy * u and the product.
    tol = lead * OA.slope_error(zz, act) + 2 * U * np.abs(dz) + 2.0 ** -149
    assert_codes(r.dz, dz * scale, tol * scale + U * np.abs(dz * scale), fmt, "dz")
    assert_folded(before, ring, float(np.max(np.abs(dz), initial=0.0)), float(np.max(tol, initial=0.0)), fmt)
    if db:
        _sums(r.db, dz.sum(0), dz, tol, "db")
    else:
        assert r.db is None
    if u is None:
        assert r.du is None and r.dbu is None
        return r
    tol = np.abs(d) * OA.value_error(zz, act) + U * np.abs(du) + 2.0 ** -149
    assert_codes(r.du, du * scale / 2, tol * scale + U * np.abs(du * scale), fmt, "du")
    assert_folded(before_u, ring_u, float(np.max(np.abs(du), initial=0.0)), float(np.max(tol, initial=0.0)), fmt)
    if db:
        _sums(r.dbu, du.sum(0), du, tol, "dbu")
    return r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_act_backward(rows, cols, dtype):
    for k, act in enumerate(ACTS):
        for gate in (False, True):
            dy, z, u = _inputs(rows, cols, dtype, rows + cols + k, gate)
            _check(dy, z, u, act, ops.E5M2, True)
            _check(dy, z, u, act, ops.E4M3, False)


@pytest.mark.parametrize("db", [False, True])
@pytest.mark.parametrize("offset", [1, 3, 4])
@pytest.mark.parametrize("cols", [8, 1024, 1537])
def test_act_backward_at_any_element_alignment(cols, offset, db):
    for dtype in ("bf16", "fp32"):
        dy, z, u = _inputs(50, cols, dtype, cols, True)
        _check(dy, z, u, ops.ACT_SILU, ops.E5M2, db, offset)


def test_act_backward_training_sized_repeats_its_bits():
    dy, z, u = _inputs(4096, 1536, "bf16", 1, True)
    a = _check(dy, z, u, ops.ACT_SILU, ops.E5M2, True)
    b = _check(dy, z, u, ops.ACT_SILU, ops.E5M2, True)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    c = _check(dy, z, u, ops.ACT_SILU, ops.E5M2, False)
    assert torch.equal(a.dz, c.dz) and torch.equal(a.du, c.du)


def test_act_backward_tall_and_wide():
    _check(*_inputs(20000, 24, "bf16", 2, False), ops.ACT_GELU, ops.E5M2, True)
    _check(*_inputs(2, 70000, "bf16", 3, True), ops.ACT_RELU, ops.E5M2, True)


def test_cast_with_bias_gradient_is_quantize_and_bias_grad():
    dy, _, _ = _inputs(300, 1536, "bf16", 4, False)
    r = _check(dy, None, None, ops.ACT_NONE, ops.E5M2, True)
    ring = ops.Ring(scale=30.0)
    codes, _ = ops.quantize(dy.cuda(), ops.E5M2, ops.ROW, ring)
    assert torch.equal(codes, r.dz)


def test_act_backward_of_huge_and_special_pre_activations():
    z = torch.tensor([[0.0, -0.0, 1e-30, 200.0, -200.0, 3e38, -3e38, 1e25, -1e25, float("nan")]], dtype=torch.bfloat16)
    dy = torch.ones(1, 10, dtype=torch.float32)
    want = {ops.ACT_RELU: [0, 0, 1, 1, 0, 1, 0, 1, 0], ops.ACT_SILU: [.5, .5, .5, 1, 0, 1, 0, 1, 0],
            ops.ACT_GELU: [.5, .5, .5, 1, 0, 1, 0, 1, 0]}
    for act, w in want.items():
        ring = ops.Ring()
        r = ops.act_backward(dy.cuda(), z.cuda(), act, ops.E4M3, ring)
        got = r.dz.view(torch.float8_e4m3fn).float().cpu()[0]
        assert got[:9].tolist() == w, act
        assert float(ring.state()[0][0]) == 1.0  # a NaN does not enter the amax


def test_relu_lets_nothing_through_where_it_is_zero():
    """Infinite and NaN gradients (and gates) where z <= 0 reach neither dz, nor its amax, nor the sums."""
    bad = float("inf"), float("-inf"), float("nan")
    z = torch.tensor([[-1.0, -0.0, 0.0, 2.0]] * 3, dtype=torch.bfloat16)
    for db in (False, True):
        for gate in (False, True):
            dy = torch.tensor([[b, b, b, 1.0] for b in bad], dtype=torch.bfloat16)
            u = torch.tensor([[b, b, b, 3.0] for b in bad[::-1]], dtype=torch.bfloat16) if gate else None
            ring, ring_u = ops.Ring(), ops.Ring() if gate else None
            r = ops.act_backward(dy.cuda(), z.cuda(), ops.ACT_RELU, ops.E4M3, ring, None if u is None else u.cuda(),
                                 ring_u, need_db=db)
            got = r.dz.view(torch.float8_e4m3fn).float().cpu()
            assert got.tolist() == [[0, 0, 0, 3.0 if gate else 1.0]] * 3
            assert float(ring.state()[0][0]) == (3.0 if gate else 1.0)
            assert not db or r.db.tolist() == [0, 0, 0, 9.0 if gate else 3.0]


@pytest.mark.parametrize("db", [False, True])
def test_act_backward_offsets_beyond_31_bits(db):
    rows, cols = 70000, 32768  # 2.29e9 elements
    tail = _inputs(3, cols, "bf16", 5, False)
    dy, z = (torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dy[-3:].copy_(tail[0])
    z[-3:].copy_(tail[1])
    ring = ops.Ring(scale=30.0)
    r = ops.act_backward(dy, z, ops.ACT_SILU, ops.E5M2, ring, need_db=db)
    want = ops.act_backward(dy[-3:].clone(), z[-3:].clone(), ops.ACT_SILU, ops.E5M2, ops.Ring(scale=30.0), need_db=db)
    torch.cuda.synchronize()
    assert torch.equal(r.dz[-3:], want.dz) and not r.dz[:3].any() and not r.dz[-6:-3].any()
    if db:  # the zeros add nothing
        assert_within(f64(r.db), f64(want.db), 4 * U * np.abs(f64(tail[0])).sum(0) * 1.2, "db")


def test_act_backward_empty_batch():
    for u, ring_u in ((None, None), (torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"), ops.Ring(scale=3.0))):
        ring = ops.Ring(scale=2.0)
        before = ring.state()
        e = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
        r = ops.act_backward(e, e, ops.ACT_SILU, ops.E5M2, ring, u, ring_u, need_db=True)
        assert r.dz.shape == (0, 40) and not r.db.any() and r.db.shape == (40,)
        assert_folded(before, ring, 0.0, 0.0, ops.E5M2)
        assert ring_u is None or (ring_u.state()[1] == 1 and not r.dbu.any())


def test_act_backward_shards_leave_the_fold_to_the_ranks():
    dy, z, u = (t.cuda() for t in _inputs(64, 512, "bf16", 10, True))
    whole, whole_u, shard, shard_u = (ops.Ring(scale=5.0) for _ in range(4))
    want = ops.act_backward(dy, z, ops.ACT_SILU, ops.E5M2, whole, u, whole_u)
    ams = []
    for p in (slice(0, 24), slice(24, 64)):
        a = torch.zeros(2, device="cuda")
        got = ops.act_backward(dy[p], z[p], ops.ACT_SILU, ops.E5M2, shard, u[p], shard_u, amax=a[:1], amax_u=a[1:])
        assert torch.equal(got.dz, want.dz[p]) and torch.equal(got.du, want.du[p])
        ams.append(a)
    m = torch.maximum(*ams)
    ops.ring_fold(shard, ops.E5M2, m[:1])
    ops.ring_fold(shard_u, ops.E5M2, m[1:])
    torch.cuda.synchronize()
    assert torch.equal(whole.buf, shard.buf) and torch.equal(whole_u.buf, shard_u.buf)


def test_act_backward_on_another_stream_and_in_two_graphs():
    dy, z, u = (t.cuda() for t in _inputs(512, 1024, "bf16", 11, True))
    want = ops.act_backward(dy, z, ops.ACT_GELU, ops.E5M2, ops.Ring(), u, ops.Ring(), need_db=True)
    s = torch.cuda.Stream()
    rings = ops.Ring(), ops.Ring()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.act_backward(dy, z, ops.ACT_GELU, ops.E5M2, rings[0], u, rings[1], need_db=True, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graphs = []
    for k in range(2):
        rk, dk = (ops.Ring(), ops.Ring()), dy * (k + 1)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ops.act_backward(dk, z, ops.ACT_GELU, ops.E5M2, rk[0], u, rk[1], need_db=True)
        graphs.append((g, rk, dk, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        for st, (g, *_rest) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for g, rk, dk, out in graphs:
        r2 = ops.Ring(), ops.Ring()
        for _ in range(2):
            o2 = ops.act_backward(dk, z, ops.ACT_GELU, ops.E5M2, r2[0], u, r2[1], need_db=True)
        torch.cuda.synchronize()
        for a, b in zip(out, o2):
            assert torch.equal(a, b)
        assert torch.equal(rk[0].buf, r2[0].buf) and torch.equal(rk[1].buf, r2[1].buf)


def test_act_backward_refuses_what_the_binding_can_see():
    dy, z, u = (t.cuda() for t in _inputs(4, 16, "bf16", 0, True))
    ring = ops.Ring()
    for call in (lambda: ops.act_backward(dy.cpu(), z, 1, 1, ring), lambda: ops.act_backward(dy, z.float(), 1, 1, ring),
                 lambda: ops.act_backward(dy, z[:2], 1, 1, ring), lambda: ops.act_backward(dy.t(), z, 1, 1, ring),
                 lambda: ops.act_backward(dy, z, 1, 1, ring, u), lambda: ops.act_backward(dy, z, 1, 1, ring, None, ring),
                 lambda: ops.act_backward(dy.long(), z, 1, 1, ring)):
        with pytest.raises(ValueError):
            call()
    for args in ((dy, z, 4, 1, ring), (dy, z, 1, 2, ring), (dy, None, 1, 1, ring), (dy, z, 1, 1, ring, u, ring)):
        with pytest.raises(ops.Fp8Error) as e:
            ops.act_backward(*args)
        assert e.value.status == ops.FP8_ERR_INVALID_ARG
