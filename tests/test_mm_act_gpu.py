"""GPU parity of the product with an activation epilogue against the oracle."""

import numpy as np
import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops, synthetic as S
from gpu_helpers import OF, OG, band_rows, require_gpu
from layer_helpers import HALF, U, assert_codes, assert_folded, assert_within, at_offset, f64
from oracle import act as OA

pytestmark = pytest.mark.gpu

ACTS = [ops.ACT_NONE, ops.ACT_RELU, ops.ACT_GELU, ops.ACT_SILU]
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _codes(shape, seed, fmt):
    """Codes of N(0, 1) values: the products' sums stay a few units, where the activations bend."""
    v = torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    t = torch.float8_e5m2 if fmt == ops.E5M2 else torch.float8_e4m3fn
    return v.to(t).view(torch.uint8)


def _problem(M, N, K, seed, fmt_a=ops.E4M3, fmt_b=ops.E4M3, rows=False, bias=True, aux=True):
    g = torch.Generator().manual_seed(seed)
    p = dict(a=_codes((M, K), seed, fmt_a), b=_codes((N, K), seed + 1, fmt_b), fmt_a=fmt_a, fmt_b=fmt_b,
             sinv_a=torch.rand(M, generator=g) + 0.5 if rows else torch.tensor([0.75]),
             sinv_b=torch.tensor([2.0 / max(K, 1) ** 0.5]), bias=torch.randn(N, generator=g) if bias else None,
             aux=torch.randn(M, N, generator=g).to(BF) if aux else None)
    return p


def _reference(p, act, aux_op, pick):
    """(z, its tolerance, y, its tolerance) of the rows in ``pick``."""
    a, b = OF.decode(p["a"].numpy()[pick], p["fmt_a"]), OF.decode(p["b"].numpy(), p["fmt_b"])
    s = f64(p["sinv_a"]) * f64(p["sinv_b"])
    s = s[pick][:, None] if s.size > 1 else s[0]
    z = (a @ b.T) * s + (f64(p["bias"]) if p["bias"] is not None else 0.0)
    # The framework's bound on its float32 epilogue value, and the product of the two scales rounding once.
    tz = OG.bound_f32(z, (np.abs(a) @ np.abs(b).T) * s) + U * np.abs(z)
    y = OA.act(z, act)
    if act == ops.ACT_RELU:
        ty = np.where(np.abs(z) <= tz, tz, OA.slope(z, act) * tz)  # exact on either side of the kink
    else:  # Taylor: the curvature of gelu and silu stays below 2
        ty = np.abs(OA.slope(z, act)) * tz + tz * tz + OA.value_error(z, act)
    if p["aux"] is not None:
        x = f64(p["aux"])[pick]
        y, ty = (y * x, ty * np.abs(x)) if aux_op == ops.AUX_MUL else (y + x, ty)
        ty = ty + U * np.abs(y)
    return z, tz, y, ty + 2.0 ** -149


def _run(p, act, aux_op=ops.AUX_ADD, out_fmt=None, ring=None, offset=0, **kw):
    dev = {k: None if p[k] is None else p[k].cuda() for k in ("a", "b", "sinv_a", "sinv_b")}
    for k in ("bias", "aux"):
        dev[k] = None if p[k] is None else at_offset(p[k], offset)
    return ops.mm_act(dev["a"], dev["b"], dev["sinv_a"], dev["sinv_b"], act, bias=dev["bias"], aux=dev["aux"],
                      aux_op=aux_op, need_z=True, out_fmt=out_fmt, out_ring=ring, fmt_a=p["fmt_a"], fmt_b=p["fmt_b"], **kw)


def _check(p, act, aux_op=ops.AUX_ADD, out_fmt=None, offset=0, pick=None, scale=3.0, **kw):
    M = p["a"].shape[0]
    whole = pick is None
    pick = np.arange(M) if whole else pick
    z, tz, y, ty = _reference(p, act, aux_op, pick)
    ring = ops.Ring(scale=scale) if out_fmt is not None else None
    before = ring.state() if ring is not None else None
    out, zg = _run(p, act, aux_op, out_fmt, ring, offset, **kw)
    torch.cuda.synchronize()
    assert_within(f64(zg)[pick], z, tz + HALF[BF] * (np.abs(z) + tz) + 2.0 ** -134, "z")
    if out_fmt is None:
        assert_within(f64(out)[pick], y, ty + HALF[BF] * (np.abs(y) + ty) + 2.0 ** -134, "y")
        return
    assert_codes(out[torch.from_numpy(pick).cuda()], y * scale, ty * scale + U * np.abs(y * scale), out_fmt, "codes")
    if whole:
        assert_folded(before, ring, float(np.max(np.abs(y))), float(np.max(ty)), out_fmt)


# One token to a block's rows, odd widths, one k-block and a partial one.
SMALL = [(1, 1, 16), (1, 64, 1536), (2, 129, 128), (3, 4096, 48), (7, 1000, 2048), (8, 33, 4096), (9, 256, 80),
         (16, 1537, 512), (17, 40, 144), (32, 520, 1024), (33, 64, 16)]
LARGE = [(64, 257, 512), (130, 700, 512), (129, 2048, 256), (1000, 1537, 512), (300, 1536, 4096)]


@pytest.mark.parametrize("M,N,K", SMALL + LARGE)
def test_mm_act_every_activation_and_operand(M, N, K):
    for k, act in enumerate(ACTS):
        for aux in (None, ops.AUX_ADD, ops.AUX_MUL):
            p = _problem(M, N, K, 7 * M + k, rows=(k + (aux or 0)) % 2 == 0, bias=k % 2 == 0, aux=aux is not None)
            _check(p, act, aux or 0, None)
            _check(p, act, aux or 0, ops.E4M3 if k % 2 else ops.E5M2)


@pytest.mark.parametrize("fmt_a", [ops.E4M3, ops.E5M2])
@pytest.mark.parametrize("fmt_b", [ops.E4M3, ops.E5M2])
@pytest.mark.parametrize("M", [1, 12, 200])
def test_mm_act_operand_formats(M, fmt_a, fmt_b):
    _check(_problem(M, 320, 256, 3, fmt_a, fmt_b, rows=True), ops.ACT_GELU, ops.AUX_ADD, ops.E4M3)


@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("N", [256, 264, 260, 257])
def test_mm_act_at_any_element_alignment(M, N):
    p = _problem(M, N, 256, N, rows=True)
    for out_fmt in (None, ops.E4M3):
        shape = (M, N)
        flat = torch.zeros(M * N + 5, dtype=BF if out_fmt is None else torch.uint8, device="cuda")
        zflat = torch.zeros(M * N + 3, dtype=BF, device="cuda")
        _check(p, ops.ACT_SILU, ops.AUX_MUL, out_fmt, offset=1, out=flat[3:-2].view(shape), z=zflat[1:-2].view(shape))
        assert not flat[:3].any() and not flat[-2:].any() and not zflat[:1].any() and not zflat[-2:].any()


# (256-wide tiles on CTA pairs) and the other shapes the chooser has, in training sizes.
@pytest.mark.parametrize("M,N,K,act,aux_op,out_fmt", [
    (2048, 4096, 1536, ops.ACT_SILU, ops.AUX_MUL, ops.E4M3),
    (2048, 1536, 4096, ops.ACT_NONE, ops.AUX_ADD, None),
    (1536, 1537, 2048, ops.ACT_GELU, ops.AUX_ADD, ops.E4M3),
    (512, 4096, 1536, ops.ACT_RELU, ops.AUX_ADD, None),
    (384, 8192, 1024, ops.ACT_SILU, ops.AUX_MUL, None),
])
def test_mm_act_training_sizes(M, N, K, act, aux_op, out_fmt):
    p = _problem(M, N, K, 5)
    _check(p, act, aux_op, out_fmt, pick=band_rows(M, 1))


@pytest.mark.parametrize("out_fmt,N", [(None, 32768), (ops.E4M3, 32768), (ops.E4M3, 32769)])
def test_mm_act_offsets_beyond_31_bits(out_fmt, N):
    """2.29e9 outputs; direct, staged and guarded stores."""
    M, K = 70000, 16
    p = _problem(128, N, K, 11, aux=False)
    a = p["a"].repeat((M + 127) // 128, 1)[:M].contiguous().cuda()
    b, sa, sb, bias = (p[k].cuda() for k in ("b", "sinv_a", "sinv_b", "bias"))
    ring, ring2 = (ops.Ring(scale=3.0) if out_fmt is not None else None for _ in range(2))
    out, _ = ops.mm_act(a, b, sa, sb, ops.ACT_GELU, bias=bias, out_fmt=out_fmt, out_ring=ring)
    want, _ = ops.mm_act(a[:128].contiguous(), b, sa, sb, ops.ACT_GELU, bias=bias, out_fmt=out_fmt, out_ring=ring2)
    torch.cuda.synchronize()
    for m in (0, 128, 65536, M // 128 * 128 - 128):  # rows repeat every 128
        assert torch.equal(out[m:m + 128], want), m
    last = M // 128 * 128
    assert torch.equal(out[last:], want[:M - last])


@pytest.mark.parametrize("M,N,aux", [(128, 256, False), (128, 256, True), (600, 1024, True), (600, 1000, True),
                                     (2000, 1024, True), (2000, 1000, True)])
def test_mm_act_wait_runs_out_then_the_next_call_is_right(M, N, aux):
    """The timeout path (see the timeout tests of the product): the stopped kernel lets its
    operand loads land, frees what it holds and returns; the next call is whole."""
    p = _problem(M, N, 4096, 12, aux=aux)
    torch.cuda.synchronize()
    assert ops.device_error(clear=True)[0] == ops.FP8_OK
    ops.debug_wait(20_000, ops.SITE_EPILOGUE_TMEM_FULL)
    try:
        _run(p, ops.ACT_SILU, ops.AUX_MUL, ops.E4M3, ops.Ring())
        torch.cuda.synchronize()
    finally:
        ops.debug_wait()
    rc, where = ops.device_error(clear=True)
    assert rc == ops.FP8_ERR_DEVICE_TIMEOUT and where == ops.SITE_EPILOGUE_TMEM_FULL, (rc, where)
    _check(p, ops.ACT_SILU, ops.AUX_MUL, ops.E4M3)


def test_mm_act_without_anything_is_mm():
    """No activation, no operand: bit for bit the framework's product, where both take the tile kernel."""
    for M, N, K in ((300, 512, 256), (1000, 1537, 512)):
        p = _problem(M, N, K, 1, aux=False)
        out, z = _run(p, ops.ACT_NONE)
        ref = ops.mm(p["a"].cuda(), p["b"].cuda(), p["sinv_a"].cuda(), p["sinv_b"].cuda(), p["bias"].cuda())
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(z, ref)


@pytest.mark.parametrize("M", [1, 40])
def test_mm_act_residual_in_place(M):
    p = _problem(M, 512, 256, 2)
    want, _ = _run(p, ops.ACT_RELU)
    x = p["aux"].cuda()
    got, _ = ops.mm_act(p["a"].cuda(), p["b"].cuda(), p["sinv_a"].cuda(), p["sinv_b"].cuda(), ops.ACT_RELU,
                        bias=p["bias"].cuda(), aux=x, out=x)
    torch.cuda.synchronize()
    assert got is x and torch.equal(x, want)


@pytest.mark.parametrize("M", [3, 50])
def test_mm_act_k0_and_empty(M):
    p = _problem(M, 96, 0, 4)
    for out_fmt in (None, ops.E5M2):
        _check(p, ops.ACT_SILU, ops.AUX_MUL, out_fmt)
    ring = ops.Ring(scale=2.0)
    before = ring.state()
    e = torch.empty(0, 64, dtype=torch.uint8, device="cuda")
    s = torch.ones(1, device="cuda")
    out, z = ops.mm_act(e, _codes((32, 64), 1, 0).cuda(), s, s, ops.ACT_SILU, out_fmt=ops.E4M3, out_ring=ring, need_z=True)
    assert out.shape == (0, 32) and z.shape == (0, 32)
    assert_folded(before, ring, 0.0, 0.0, ops.E4M3)


@pytest.mark.parametrize("M", [2, 70])
def test_mm_act_nan_and_infinity_stay_in_their_rows(M):
    p = _problem(M, 200, 128, 6, aux=False)
    p["a"][0, 3] = 0x7F  # NaN
    out, z = _run(p, ops.ACT_GELU)
    assert torch.isnan(out[0]).all() and torch.isnan(z[0]).all() and torch.isfinite(out[1:]).all()
    p["a"][0, 3] = 0
    p["bias"][5], p["bias"][6] = float("inf"), 1e30
    out, z = _run(p, ops.ACT_SILU)
    assert torch.isinf(out[:, 5]).all() and torch.isfinite(out[:, 6]).all() and torch.isfinite(out[:, 7:]).all()


@pytest.mark.parametrize("M", [8, 96])
def test_mm_act_shards_leave_the_fold_to_the_ranks(M):
    p = _problem(M, 512, 256, 8)
    d = {k: p[k].cuda() for k in ("a", "b", "sinv_a", "sinv_b", "bias", "aux")}
    args = (d["b"], d["sinv_a"], d["sinv_b"], ops.ACT_SILU)
    # Shards of one size class, so that both take the whole call's kernel.
    whole, shard = ops.Ring(scale=5.0), ops.Ring(scale=5.0)
    want, _ = ops.mm_act(d["a"], *args, bias=d["bias"], aux=d["aux"], out_fmt=ops.E4M3, out_ring=whole)
    ams = []
    for s in (slice(0, M // 2), slice(M // 2, M)):
        a = torch.zeros(1, device="cuda")
        got, _ = ops.mm_act(d["a"][s], *args, bias=d["bias"], aux=d["aux"][s], out_fmt=ops.E4M3, out_ring=shard,
                            out_amax=a)
        assert torch.equal(got, want[s])
        ams.append(a)
    ops.ring_fold(shard, ops.E4M3, torch.maximum(*ams))
    torch.cuda.synchronize()
    assert torch.equal(whole.buf, shard.buf)


@pytest.mark.parametrize("M", [4, 256])
def test_mm_act_on_another_stream_and_in_two_graphs(M):
    p = _problem(M, 1024, 512, 9)
    d = {k: p[k].cuda() for k in ("a", "b", "sinv_a", "sinv_b", "bias", "aux")}

    def call(a, ring, **kw):
        return ops.mm_act(a, d["b"], d["sinv_a"], d["sinv_b"], ops.ACT_GELU, bias=d["bias"], aux=d["aux"], need_z=True,
                          out_fmt=ops.E4M3, out_ring=ring, **kw)

    want = call(d["a"], ops.Ring(scale=2.0))
    s = torch.cuda.Stream()
    ring = ops.Ring(scale=2.0)
    s.wait_stream(torch.cuda.current_stream())
    got = call(d["a"], ring, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs = []
    for k in range(2):
        rk, ak = ops.Ring(scale=2.0), d["a"] if k == 0 else d["a"].flip(0).contiguous()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(ak, rk)
        graphs.append((g, rk, ak, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, (g, *_rest) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for g, rk, ak, out in graphs:
        r2 = ops.Ring(scale=2.0)
        for _ in range(3):
            o2 = call(ak, r2)
        torch.cuda.synchronize()
        assert torch.equal(out[0], o2[0]) and torch.equal(out[1], o2[1]) and torch.equal(rk.buf, r2.buf)


def test_mm_act_refuses_what_the_binding_can_see():
    p = _problem(4, 32, 64, 0)
    a, b, sa, sb, bias, aux = (p[k].cuda() for k in ("a", "b", "sinv_a", "sinv_b", "bias", "aux"))
    for call in (lambda: ops.mm_act(a.cpu(), b, sa, sb), lambda: ops.mm_act(a.float(), b, sa, sb),
                 lambda: ops.mm_act(a, b[:, :32], sa, sb), lambda: ops.mm_act(a[:, ::2], b[:, ::2], sa, sb),
                 lambda: ops.mm_act(a, b, sa.expand(3).contiguous(), sb), lambda: ops.mm_act(a, b, sa, sb.double()),
                 lambda: ops.mm_act(a, b, sa, sb, bias=bias[:4]), lambda: ops.mm_act(a, b, sa, sb, aux=aux.float()),
                 lambda: ops.mm_act(a, b, sa, sb, aux=aux.t()), lambda: ops.mm_act(a, b, sa, sb, out_fmt=ops.E4M3),
                 lambda: ops.mm_act(a, b, sa, sb, out_ring=ops.Ring()), lambda: ops.mm_act(a, b, sa, sb, out=aux[:2]),
                 lambda: ops.mm_act(a[None], b, sa, sb)):
        with pytest.raises(ValueError):
            call()
    for kw, status in ((dict(act=4), ops.FP8_ERR_INVALID_ARG), (dict(aux=aux, aux_op=2), ops.FP8_ERR_INVALID_ARG),
                       (dict(out_fmt=2, out_ring=ops.Ring()), ops.FP8_ERR_INVALID_ARG),
                       (dict(aux=aux, z=aux), ops.FP8_ERR_INVALID_ARG)):
        with pytest.raises(ops.Fp8Error) as e:
            ops.mm_act(a, b, sa, sb, **kw)
        assert e.value.status == status
    with pytest.raises(ops.Fp8Error) as e:
        ops.mm_act(a[:, :24].contiguous(), b[:, :24].contiguous(), sa, sb)
    assert e.value.status == ops.FP8_ERR_UNSUPPORTED


@pytest.mark.parametrize("N", [193, 196, 202, 255])
@pytest.mark.parametrize("out_fmt", [None, ops.E5M2])
def test_mm_act_odd_pitches_leave_the_neighbours(N, out_fmt):
    """Rows that start at every alignment, outputs inside larger buffers: nothing beyond them is written."""
    M, pad = 150, 61  # bases 2 bytes (codes: 1) off the 16-byte grid
    p = _problem(M, N, 128, N, rows=True)
    d = {k: p[k].cuda() for k in ("a", "b", "sinv_a", "sinv_b", "bias", "aux")}
    want, want_z = ops.mm_act(d["a"], d["b"], d["sinv_a"], d["sinv_b"], ops.ACT_SILU, d["bias"], d["aux"], ops.AUX_MUL,
                              need_z=True, out_fmt=out_fmt, out_ring=None if out_fmt is None else ops.Ring(scale=3.0))
    dtype = torch.bfloat16 if out_fmt is None else torch.uint8
    bufs = [torch.full((M * N + 2 * pad,), 7, dtype=t, device="cuda") for t in (dtype, torch.bfloat16, torch.bfloat16)]
    out, z, aux = (b[pad:pad + M * N].view(M, N) for b in bufs)
    aux.copy_(d["aux"])
    if out_fmt is None:
        out, bufs[0] = aux, bufs[2]  # in place
    ops.mm_act(d["a"], d["b"], d["sinv_a"], d["sinv_b"], ops.ACT_SILU, d["bias"], aux, ops.AUX_MUL, out_fmt=out_fmt,
               out_ring=None if out_fmt is None else ops.Ring(scale=3.0), out=out, z=z)
    assert torch.equal(out, want) and torch.equal(z, want_z)
    for b in bufs:
        assert bool((b[:pad] == 7).all()) and bool((b[pad + M * N:] == 7).all())
    _check(p, ops.ACT_SILU, ops.AUX_MUL, out_fmt)


# Few tiles and long K: the CTAs of a cluster share a tile's K, in equal and unequal parts.
@pytest.mark.parametrize("M,N,K", [(33, 64, 4096), (24, 512, 4096), (64, 1536, 4096), (100, 1000, 4096), (129, 1537, 4000),
                                   (256, 1536, 4096), (512, 1536, 4096), (65, 130, 16000), (40, 8, 2048), (128, 4096, 1536),
                                   (48, 520, 1040), (100, 96, 656)])
def test_mm_act_few_tiles_and_long_k(M, N, K):
    for k, (act, aux, out_fmt) in enumerate(((ops.ACT_SILU, ops.AUX_MUL, ops.E4M3), (ops.ACT_GELU, ops.AUX_ADD, None),
                                             (ops.ACT_RELU, None, ops.E5M2))):
        p = _problem(M, N, K, 31 * M + k, rows=k == 0, bias=k != 1, aux=aux is not None)
        _check(p, act, aux or ops.AUX_ADD, out_fmt)
        runs = [_run(p, act, aux or ops.AUX_ADD, out_fmt, None if out_fmt is None else ops.Ring(scale=3.0)) for _ in range(3)]
        for out, z in runs[1:]:  # the same bits in every call
            assert torch.equal(out, runs[0][0]) and torch.equal(z, runs[0][1])


def test_mm_act_few_tiles_twice_at_a_time_and_captured():
    p = _problem(96, 1536, 4096, 77, rows=True)
    want = _run(p, ops.ACT_SILU, ops.AUX_MUL, ops.E4M3, ops.Ring(scale=3.0))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for s, o in zip(streams, outs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                o.append(_run(p, ops.ACT_SILU, ops.AUX_MUL, ops.E4M3, ops.Ring(scale=3.0)))
    torch.cuda.synchronize()
    for o in outs:
        for out, z in o:
            assert torch.equal(out, want[0]) and torch.equal(z, want[1])
    d = {k: p[k].cuda() for k in ("a", "b", "sinv_a", "sinv_b", "bias", "aux")}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, z = ops.mm_act(d["a"], d["b"], d["sinv_a"], d["sinv_b"], ops.ACT_SILU, d["bias"], d["aux"], ops.AUX_MUL,
                            need_z=True)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, want[1])
