"""The operators in one run, as a model calls them: a gated feed-forward block between two
points of a residual stream, trained for several steps and decoded token by token.

    h = x + residual;  n = rmsnorm(h);  u = n Wu^T;  a = silu(n Wg^T) * u;  y = h + a Wd^T

Against the same block in float64 without any rounding.  Rounding to E4M3 is off by at most
2^-4 relative, and evenly spread below that: 2^-4 / sqrt(3) in the mean square, E5M2 twice as
much.  A result's relative error (2-norm) is at most the sum of those of the casts on the way
to it, each weighted with the slope that it meets; no slope of silu exceeds 1.1.  bf16
roundings (2^-8) add a few hundredths of that.
"""

import numpy as np
import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

Q4, Q5 = 2.0 ** -4 / 3 ** 0.5, 2.0 ** -3 / 3 ** 0.5
D, F, EPS = 256, 640, 1e-6


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _model(seed):
    g = torch.Generator().manual_seed(seed)
    p = dict(gamma=1 + 0.1 * torch.randn(D, generator=g), wg=torch.randn(F, D, generator=g) / 16,
             wu=torch.randn(F, D, generator=g) / 16, wd=torch.randn(D, F, generator=g) / 25)
    return {k: v.to(torch.bfloat16) for k, v in p.items()}


def _tokens(M, seed):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(M, D, generator=g).to(torch.bfloat16) for _ in range(3))  # x, residual, dy


def _exact(p, x, res, dy):
    """(y, gradients) in float64; h rounded as the stream keeps it."""
    w = {k: v.double().requires_grad_() for k, v in p.items()}
    h = (x.float() + res.float()).to(torch.bfloat16).double().requires_grad_()
    n = h * (h.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * w["gamma"]
    y = h + (torch.nn.functional.silu(n @ w["wg"].t()) * (n @ w["wu"].t())) @ w["wd"].t()
    y.backward(dy.double())
    return y.detach(), dict({k: v.grad for k, v in w.items()}, x=h.grad), h.detach()


class Block:
    """The block's rings and one training step of it through the framework's calls."""

    def __init__(self, p):
        self.p = {k: v.cuda() for k, v in p.items()}
        self.r = {k: ops.Ring() for k in ("n", "wg", "wu", "wd", "a", "dy", "dz", "du")}

    def weights(self):
        r = self.r
        q = ops.quantize_multi([dict(x=self.p[k], fmt=ops.E4M3, layout=ops.ROW, ring=r[k]) for k in ("wg", "wu", "wd")])
        return [c for c, _ in q]

    def step(self, x, res, dy):
        r, p = self.r, self.p
        wg, wu, wd = self.weights()
        n = ops.rmsnorm(x, p["gamma"], res, eps=EPS, fmt=ops.E4M3, ring=r["n"], need_rstd=True)
        u = ops.mm(n.codes, wu, n.sinv, r["wu"].scale_inv)
        a, z = ops.mm_act(n.codes, wg, n.sinv, r["wg"].scale_inv, ops.ACT_SILU, aux=u, aux_op=ops.AUX_MUL, need_z=True,
                          out_fmt=ops.E4M3, out_ring=r["a"])
        y, _ = ops.mm_act(a, wd, r["a"].scale_inv, r["wd"].scale_inv, aux=n.h)
        # Backward: the layout tag reads row-layout codes as transposed operands.
        dyq, _ = ops.quantize(dy, ops.E5M2, ops.ROW, r["dy"])
        da, dwd = ops.mm_pair(dict(a=dyq, b=wd, sinv_a=r["dy"].scale_inv, sinv_b=r["wd"].scale_inv, fmt_a=ops.E5M2,
                                   b_mn_major=True),
                              dict(a=dyq, b=a, sinv_a=r["dy"].scale_inv, sinv_b=r["a"].scale_inv, fmt_a=ops.E5M2,
                                   a_mn_major=True, b_mn_major=True))
        g = ops.act_backward(da, z, ops.ACT_SILU, ops.E5M2, r["dz"], u, r["du"])
        dn, grads = None, {}
        for k, c, ring, w in (("wg", g.dz, r["dz"], wg), ("wu", g.du, r["du"], wu)):
            d, grads[k] = ops.mm_pair(dict(a=c, b=w, sinv_a=ring.scale_inv, sinv_b=r[k].scale_inv, fmt_a=ops.E5M2,
                                           b_mn_major=True),
                                      dict(a=c, b=n.codes, sinv_a=ring.scale_inv, sinv_b=n.sinv, fmt_a=ops.E5M2,
                                           a_mn_major=True, b_mn_major=True))
            dn = d if dn is None else dn + d
        dx, dgamma = ops.rmsnorm_backward(dn, n.h, n.rstd, p["gamma"], dres=dy)
        return y, dict(grads, wd=dwd, gamma=dgamma, x=dx), n.h


def _off(got, ref):
    got, ref = got.double().cpu(), ref.double()
    return float((got - ref).norm() / ref.norm())


def test_training_steps_against_float64():
    p = _model(0)
    blk = Block(p)
    M = 320
    for step in range(4):  # the first on scale 1, the others on delayed scales
        x, res, dy = _tokens(M, 10 + step)
        y, grads, h = blk.step(x.cuda(), res.cuda(), dy.cuda())
        torch.cuda.synchronize()
        y_ref, ref, h_ref = _exact(p, x, res, dy)
        assert torch.equal(h.cpu().double(), h_ref)
        if step == 0:
            continue  # scale 1 leaves most gradients below E5M2's normal range
        bf = 2.0 ** -8
        act = 2 * Q4 * 1.1 + 2 * Q4  # what silu(gate) * up carries: n and wg, n and wu
        assert _off(y.cpu().double() - h_ref, y_ref - h_ref) < act + Q4 + Q4 + 4 * bf  # + a's cast, wd
        # The gradient of a: dy and wd; of z and u: that, the other factor's error, the slope's, the cast.
        da = Q5 + Q4
        dz = da + act + 2 * Q4 + Q5
        bounds = dict(wd=Q5 + act + Q4, wg=dz + Q4, wu=dz + Q4, x=dz + Q4 + 2 * bf, gamma=dz + Q4 + 2 * bf)
        for k, b in bounds.items():
            if k == "x":  # the residual stream's own gradient is exact: the branch's error is measured
                assert _off(grads[k].cpu().double() - dy.double(), ref[k] - dy.double()) < b + 4 * bf, k
            else:
                assert _off(grads[k], ref[k]) < b + 4 * bf, k


def test_training_step_in_a_graph_is_the_eager_step():
    p = _model(1)
    x, res, dy = (t.cuda() for t in _tokens(256, 3))
    eager, graphed = Block(p), Block(p)
    graphed.step(x, res, dy)  # tensor maps and first-call set-up before the capture
    for k in graphed.r:
        graphed.r[k].buf.copy_(ops.Ring().buf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = graphed.step(x, res, dy)
    for _ in range(3):
        want = eager.step(x, res, dy)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0])
    for k in out[1]:
        assert torch.equal(out[1][k], want[1][k]), k
    for k in eager.r:
        assert torch.equal(eager.r[k].buf, graphed.r[k].buf), k


@pytest.mark.parametrize("M", [1, 5, 24, 40])
def test_decoding_with_row_scales(M):
    """Serving keeps no state: rows scale themselves, the activation has its calibrated ring."""
    p = _model(2)
    x, res, dy = _tokens(M, 4)
    blk = Block(p)
    for _ in range(2):
        wg, wu, wd = blk.weights()
    a_ring = ops.Ring(scale=448.0 / 40.0)
    amax = torch.zeros(1, device="cuda")
    frozen = a_ring.buf.clone()
    n = ops.rmsnorm(x.cuda(), blk.p["gamma"], res.cuda(), eps=EPS, fmt=ops.E4M3)
    u, _ = ops.mm_act(n.codes, wu, n.sinv, blk.r["wu"].scale_inv)
    a, _ = ops.mm_act(n.codes, wg, n.sinv, blk.r["wg"].scale_inv, ops.ACT_SILU, aux=u, aux_op=ops.AUX_MUL,
                      out_fmt=ops.E4M3, out_ring=a_ring, out_amax=amax)
    y, _ = ops.mm_act(a, wd, a_ring.scale_inv, blk.r["wd"].scale_inv, aux=n.h)
    torch.cuda.synchronize()
    assert torch.equal(a_ring.buf[:18], frozen[:18])  # history, idx and scale as they were
    assert 0 < float(amax) < 40.0                     # nothing saturated
    y_ref, _, h_ref = _exact(p, x, res, dy)
    # Few values: the casts' mean square is no longer sure; their largest error, sqrt(3) times it, is.
    bound = 3 ** 0.5 * (2 * Q4 * 1.1 + 2 * Q4 + 2 * Q4) + 4 * 2.0 ** -8
    assert _off(y.cpu().double() - h_ref, y_ref - h_ref) < bound
    # The same tokens one at a time.
    for m in range(min(M, 3)):
        n1 = ops.rmsnorm(x[m:m + 1].cuda(), blk.p["gamma"], res[m:m + 1].cuda(), eps=EPS, fmt=ops.E4M3)
        assert torch.equal(n1.codes, n.codes[m:m + 1]) and torch.equal(n1.sinv, n.sinv[m:m + 1])


def test_two_blocks_at_the_same_time():
    """Two streams, two blocks: nothing of one call reaches another."""
    p = _model(3)
    data = [tuple(t.cuda() for t in _tokens(192, 20 + k)) for k in range(2)]
    want = []
    for k in range(2):
        b = Block(p)
        for _ in range(3):
            w = b.step(*data[k])
        want.append((w, b))
    torch.cuda.synchronize()
    blocks, streams, got = [Block(p), Block(p)], [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    torch.cuda.synchronize()
    for _ in range(3):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] = blocks[k].step(*data[k])
    torch.cuda.synchronize()
    for k in range(2):
        (y, grads, _), b = want[k]
        assert torch.equal(got[k][0], y)
        for name in grads:
            assert torch.equal(got[k][1][name], grads[name]), name
        for name in b.r:
            assert torch.equal(b.r[name].buf, blocks[k].r[name].buf), name
