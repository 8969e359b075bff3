"""GPU parity of the norm with an FP8 output and of its gradient against the oracle."""

import numpy as np
import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops
from gpu_helpers import require_gpu
from layer_helpers import DTYPES, HALF, TINY, U, assert_codes, assert_folded, assert_within, at_offset, f64
from oracle import norm as ON

pytestmark = pytest.mark.gpu

EPS = 1e-6
# v = h * rstd * gamma in float32.  The sum of squares adds at most 32 values per
# thread one after the other, then 5 shuffles and 15 warps (52 roundings of a
# positive sum); 1/cols, its product, and eps: 2 more.  A root halves those 54;
# rsqrtf is within 2 ulp (4 U); the two products round once each: 27 + 4 + 2 < 36.
TOL_Y = 36 * U

SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 1537), (33, 1536), (300, 1024), (17, 4096), (1, 4100), (9, 8192),
          (3, 8200), (4, 16383), (2, 16384), (2500, 40)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _inputs(rows, cols, dtype, seed, residual=True, gamma32=False):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    x = torch.randn(rows, cols, generator=g)
    x = torch.where(torch.rand(rows, cols, generator=g) < 0.01, 30 * x, x).to(dt)
    res = torch.randn(rows, cols, generator=g).to(dt) if residual else None
    gamma = (1 + 0.2 * torch.randn(cols, generator=g)).to(torch.float32 if gamma32 else dt)
    return x, res, gamma


def _stream(x, res):
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def _check(x, res, gamma, fmt, ring=None, offset=0, eps=EPS):
    h_ref = _stream(x, res)
    y_ref, rstd_ref = ON.rmsnorm(f64(h_ref), f64(gamma), eps)
    before = ring.state() if ring is not None else None
    r = ops.rmsnorm(at_offset(x, offset), at_offset(gamma, offset), None if res is None else at_offset(res, offset),
                    eps=eps, fmt=fmt, ring=ring, need_rstd=True, need_y=True)
    torch.cuda.synchronize()
    assert torch.equal(r.h.cpu(), h_ref)
    assert_within(f64(r.rstd), rstd_ref, TOL_Y * rstd_ref, "rstd")
    tol = TOL_Y * np.abs(y_ref) + 2.0 ** -149
    assert_within(f64(r.y), y_ref, tol + HALF[x.dtype] * np.abs(y_ref) * 1.001 + TINY[x.dtype], "y")
    if ring is not None:
        s = before[2]
        assert_codes(r.codes, y_ref * s, tol * s + U * np.abs(y_ref * s), fmt, "codes")
        a = float(np.max(np.abs(y_ref))) if y_ref.size else 0.0
        assert_folded(before, ring, a, TOL_Y * a, fmt)
        assert r.sinv.item() == ring.scale_inv.item()
    else:
        s = ON.row_scales(y_ref, fmt)
        # The row's amax is off by TOL_Y, FMAX / amax and 1 / scale round once each.
        assert_within(f64(r.sinv), 1 / s, (TOL_Y + 3 * U) / s, "sinv")
        v = y_ref * s[:, None]
        assert_codes(r.codes, v, (2 * TOL_Y + 4 * U) * np.abs(v), fmt, "codes")
    return r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_rings_and_rows(rows, cols, dtype):
    x, res, gamma = _inputs(rows, cols, dtype, rows * 31 + cols)
    ring = ops.Ring(scale=3.7)
    _check(x, res, gamma, ops.E4M3, ring)
    _check(x, None, gamma, ops.E4M3, ring)  # on the scale that the first call published
    _check(x, res, gamma, ops.E5M2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("offset", [1, 3, 4])
@pytest.mark.parametrize("cols", [8, 1024, 1537, 5000])
def test_norm_at_any_element_alignment(cols, offset, dtype):
    x, res, gamma = _inputs(7, cols, dtype, cols + offset, gamma32=offset == 3)
    _check(x, res, gamma, ops.E5M2, ops.Ring(scale=100.0), offset)
    _check(x, None, gamma, ops.E4M3, None, offset)


def test_norm_long_and_training_sized():
    x, res, gamma = _inputs(8192, 1536, "bf16", 5)
    _check(x, res, gamma, ops.E4M3, ops.Ring(scale=4.0))
    x, res, gamma = _inputs(20000, 72, "fp16", 6)
    _check(x, res, gamma, ops.E4M3, ops.Ring(scale=4.0))


def test_norm_offsets_beyond_31_bits():
    rows, cols = 140000, 16384  # 2.29e9 elements, 4.6 GB of bf16
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, cols, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[-3:].copy_(tail)
    gamma = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    r = ops.rmsnorm(x, gamma, fmt=ops.E4M3, need_rstd=True)
    y_ref, rstd_ref = ON.rmsnorm(f64(tail), np.ones(cols), EPS)
    assert_within(f64(r.rstd[-3:]), rstd_ref, TOL_Y * rstd_ref, "rstd")
    v = y_ref * ON.row_scales(y_ref, ops.E4M3)[:, None]
    assert_codes(r.codes[-3:], v, (2 * TOL_Y + 4 * U) * np.abs(v), ops.E4M3, "codes")
    assert not r.codes[:100].any() and not r.codes[-100:-3].any()


def test_norm_empty_batch_folds_zero():
    ring = ops.Ring(scale=2.0)
    before = ring.state()
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    r = ops.rmsnorm(x, torch.ones(64, dtype=torch.bfloat16, device="cuda"), fmt=ops.E4M3, ring=ring)
    assert r.codes.shape == (0, 64)
    assert_folded(before, ring, 0.0, 0.0, ops.E4M3)
    assert ops.rmsnorm(x, torch.ones(64, device="cuda")).y.shape == (0, 64)


def test_norm_rows_of_zeros_infinities_and_nan():
    x = torch.randn(6, 96, generator=torch.Generator().manual_seed(2))
    x[1] = 0.0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 3.0e38
    gamma = torch.ones(96)
    r = ops.rmsnorm(x.cuda(), gamma.cuda(), fmt=ops.E4M3, need_rstd=True, need_y=True)
    y = r.y.cpu()
    assert not y[1].any() and r.sinv[1].item() == 1.0
    assert torch.isnan(y[2, 5]) and not y[2, :5].any()  # 1/sqrt(inf) = 0, and inf * 0
    assert torch.isnan(y[3]).all()                      # a NaN row stays in its row
    assert not y[4].any()                               # squares beyond float32: rstd 0
    ok = [0, 5]
    y_ref, _ = ON.rmsnorm(f64(x)[ok], f64(gamma), EPS)
    assert_within(f64(y)[ok], y_ref, (TOL_Y + U) * np.abs(y_ref) + 2.0 ** -149, "y")


def test_norm_in_place():
    x, res, gamma = _inputs(50, 1537, "bf16", 9)
    want = ops.rmsnorm(x.cuda(), gamma.cuda(), res.cuda(), fmt=ops.E4M3, need_y=True)
    for target in ("x", "residual"):
        xd, rd = x.cuda(), res.cuda()
        got = ops.rmsnorm(xd, gamma.cuda(), rd, fmt=ops.E4M3, h=xd if target == "x" else rd)
        assert torch.equal(got.h, want.h) and torch.equal(got.codes, want.codes)
        assert got.h.data_ptr() == (xd if target == "x" else rd).data_ptr()
    xd, rd = x.cuda(), res.cuda()
    got = ops.rmsnorm(xd, gamma.cuda(), rd, fmt=ops.E4M3, h=rd, y=xd)
    assert torch.equal(got.h, want.h) and torch.equal(got.y, want.y)


def test_norm_shards_leave_the_fold_to_the_ranks():
    x, res, gamma = _inputs(64, 512, "bf16", 10)
    whole, shard = ops.Ring(scale=5.0), ops.Ring(scale=5.0)
    want = ops.rmsnorm(x.cuda(), gamma.cuda(), res.cuda(), fmt=ops.E4M3, ring=whole)
    amaxes = []
    for part in (slice(0, 24), slice(24, 64)):
        a = torch.zeros(1, device="cuda")
        got = ops.rmsnorm(x[part].cuda(), gamma.cuda(), res[part].cuda(), fmt=ops.E4M3, ring=shard, amax=a)
        assert torch.equal(got.codes, want.codes[part])
        amaxes.append(a)
    ops.ring_fold(shard, ops.E4M3, torch.maximum(*amaxes))
    torch.cuda.synchronize()
    assert torch.equal(whole.buf, shard.buf)


def _check_backward(x, dy, gamma, dres, offset=0):
    h = f64(x)
    rstd = torch.from_numpy(1 / np.sqrt(np.mean(h * h, axis=1) + EPS)).float()
    dx_ref, dg_ref = ON.rmsnorm_backward(f64(dy), h, f64(rstd), f64(gamma), None if dres is None else f64(dres))
    dx, dg = ops.rmsnorm_backward(at_offset(dy, offset), at_offset(x, offset), rstd.cuda(), at_offset(gamma, offset),
                                  None if dres is None else at_offset(dres, offset))
    torch.cuda.synchronize()
    r = f64(rstd)[:, None]
    n, g = h * r, f64(dy) * f64(gamma)
    d = 0.0 if dres is None else np.abs(f64(dres))
    # mean(g n): each term rounds three times, at most 52 additions, 1/cols and its product:
    # 57 U of mean |g n|; g, n, their join and the join with dres round a few times each.
    tol = r * (4 * U * np.abs(g) + np.abs(n) * 60 * U * np.mean(np.abs(g * n), axis=1, keepdims=True)) + 2 * U * d
    assert_within(f64(dx), dx_ref, tol + HALF[x.dtype] * (np.abs(dx_ref) + tol) + TINY[x.dtype], "dx")
    # Each term rounds twice; a sum of R terms in any order at most R - 1 times.
    S = np.sum(np.abs(f64(dy) * n), axis=0)
    assert_within(f64(dg), dg_ref, (x.shape[0] + 2) * U * S + 2.0 ** -149, "dgamma")
    return dx, dg


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_backward(rows, cols, dtype):
    x, _, gamma = _inputs(rows, cols, dtype, rows + cols)
    g = torch.Generator().manual_seed(rows)
    dy = (torch.randn(rows, cols, generator=g) * 1e-2).to(x.dtype)
    dres = (torch.randn(rows, cols, generator=g) * 1e-2).to(x.dtype)
    _check_backward(x, dy, gamma, dres)
    _check_backward(x, dy, gamma, None)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("offset", [1, 3, 4])
@pytest.mark.parametrize("cols", [8, 1024, 1537, 5000])
def test_norm_backward_at_any_element_alignment(cols, offset, dtype):
    x, dres, gamma = _inputs(600, cols, dtype, cols, gamma32=offset == 1)
    dy = _inputs(600, cols, dtype, 99, residual=False)[0]
    _check_backward(x, dy, gamma, dres, offset)


def test_norm_backward_repeats_its_bits_in_place_and_on_no_rows():
    x, dres, gamma = _inputs(3000, 1536, "bf16", 3)
    dy = _inputs(3000, 1536, "bf16", 4)[0]
    dx, dg = _check_backward(x, dy, gamma, dres)
    rstd = torch.rsqrt(x.double().square().mean(1) + EPS).float().cuda()
    a = ops.rmsnorm_backward(dy.cuda(), x.cuda(), rstd, gamma.cuda(), dres.cuda())
    for target in ("dy", "dres"):
        t = dict(dy=dy.cuda(), dres=dres.cuda())
        b = ops.rmsnorm_backward(t["dy"], x.cuda(), rstd, gamma.cuda(), t["dres"], dx=t[target])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    only, none = ops.rmsnorm_backward(dy.cuda(), x.cuda(), rstd, gamma.cuda(), dres.cuda(), need_dgamma=False)
    assert none is None and torch.equal(only, a[0])
    e = torch.empty(0, 40, device="cuda")
    dx, dg = ops.rmsnorm_backward(e, e, torch.empty(0, device="cuda"), torch.ones(40, device="cuda"))
    assert dx.shape == (0, 40) and dg.shape == (40,) and not dg.any()


def test_norm_gradient_of_the_whole_call_against_autograd():
    """x and residual share one gradient; gamma's is that of every row."""
    x, res, gamma = _inputs(40, 200, "fp32", 8)
    dy = torch.randn(40, 200, generator=torch.Generator().manual_seed(1))
    xs, rs, gs = (t.double().requires_grad_() for t in (x, res, gamma))
    h = xs + rs
    (h * (h.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * gs).backward(dy.double())
    r = ops.rmsnorm(x.cuda(), gamma.cuda(), res.cuda(), need_rstd=True)
    dx, dg = ops.rmsnorm_backward(dy.cuda(), r.h, r.rstd, gamma.cuda())
    assert torch.equal(xs.grad, rs.grad)
    # float32 rounding of h (U relative) moves every factor by a few U; the sums add up to 64.
    scale = float(xs.grad.abs().max())
    assert_within(f64(dx), xs.grad.numpy(), 100 * U * scale, "dx")
    assert_within(f64(dg), gs.grad.numpy(), 100 * U * float((dy.abs() * 10).sum(0).max()), "dgamma")


def test_norm_on_another_stream_and_in_a_graph():
    x, res, gamma = (t.cuda() for t in _inputs(256, 1536, "bf16", 11))
    dy = _inputs(256, 1536, "bf16", 12)[0].cuda()
    want = ops.rmsnorm(x, gamma, res, fmt=ops.E4M3, need_rstd=True)
    want_b = ops.rmsnorm_backward(dy, want.h, want.rstd, gamma)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.rmsnorm(x, gamma, res, fmt=ops.E4M3, need_rstd=True, stream=s)
    got_b = ops.rmsnorm_backward(dy, got.h, got.rstd, gamma, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got.codes, want.codes)
    assert torch.equal(got_b[0], want_b[0]) and torch.equal(got_b[1], want_b[1])
    # Two graphs, captured one after the other, replayed in turn and at the same time.
    graphs = []
    for k in range(2):
        ring = ops.Ring(scale=2.0)
        xk = x * (k + 1)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = ops.rmsnorm(xk, gamma, res, fmt=ops.E4M3, ring=ring, need_rstd=True)
            b = ops.rmsnorm_backward(dy, r.h, r.rstd, gamma)
        graphs.append((g, ring, xk, r, b))
    refs = []
    for g, ring, xk, r, b in graphs:
        ring2 = ops.Ring(scale=2.0)
        for _ in range(3):
            r2 = ops.rmsnorm(xk, gamma, res, fmt=ops.E4M3, ring=ring2, need_rstd=True)
            b2 = ops.rmsnorm_backward(dy, r2.h, r2.rstd, gamma)
        refs.append((ring2, r2, b2))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, (g, *_rest) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (g, ring, xk, r, b), (ring2, r2, b2) in zip(graphs, refs):
        assert torch.equal(ring.buf, ring2.buf)
        assert torch.equal(r.codes, r2.codes) and torch.equal(b[0], b2[0]) and torch.equal(b[1], b2[1])


def test_norm_refuses_what_the_binding_can_see():
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(16, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: ops.rmsnorm(x.cpu(), g), lambda: ops.rmsnorm(x.t(), g), lambda: ops.rmsnorm(x, g[:8]),
                 lambda: ops.rmsnorm(x, g.half()), lambda: ops.rmsnorm(x, g, residual=x.float()),
                 lambda: ops.rmsnorm(x, g, residual=x[:, ::2]), lambda: ops.rmsnorm(x, g, h=x),
                 lambda: ops.rmsnorm(x, g, ring=ops.Ring()), lambda: ops.rmsnorm(x, g.cpu()),
                 lambda: ops.rmsnorm(x, g, fmt=ops.E4M3, amax=torch.zeros(1, device="cuda")),
                 lambda: ops.rmsnorm(x.long(), g),
                 lambda: ops.rmsnorm_backward(x, x, torch.zeros(3, device="cuda"), g)):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(fmt=2)):
        with pytest.raises(ops.Fp8Error) as e:
            ops.rmsnorm(x, g, **kw)
        assert e.value.status == ops.FP8_ERR_INVALID_ARG
