"""CPU checks of the second header: the library exports what it declares and refuses bad
arguments on the host before it touches CUDA."""

import ctypes
import os
import re

import pytest

from fp8_delayed_scaling_02_b200 import build, ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8ds_layer.h")
BAD, UNSUP = ops.FP8_ERR_INVALID_ARG, ops.FP8_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.lib()


def test_library_exports_every_declared_symbol(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fp8_[a-z_]+)\s*\(", src)))
    assert len(names) >= 3
    for name in names:
        assert hasattr(L, name), name


def _ring(addr=0x900000):
    return ops.CRing(addr, addr + 64, addr + 68, addr + 72, addr + 80)


def _norm(L, **kw):
    f = dict(x=0x100000, residual=None, dtype=0, rows=4, cols=16, gamma=0x300000, gamma_f32=0, eps=1e-6, h=None,
             y=0x500000, rstd=None, codes=None, fmt=0, ring=ops.CRing(), amax_out=None, row_sinv=None)
    f.update(kw)
    return L.fp8_rmsnorm(ctypes.byref(ops.CNormArgs(*f.values())), None)


def test_norm_refusals(L):
    assert L.fp8_rmsnorm(None, None) == BAD
    for kw in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(cols=0), dict(cols=-8), dict(eps=0.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=-1.0), dict(x=None), dict(gamma=None),
               dict(residual=0x200000), dict(h=0x400000), dict(y=None), dict(row_sinv=0x700000), dict(ring=_ring()),
               dict(codes=0x600000), dict(codes=0x600000, fmt=2, ring=_ring()),
               dict(codes=0x600000, ring=_ring(), row_sinv=0x700000),
               dict(codes=0x600000, ring=ops.CRing(0, 0, 0x900000, 0x900004, 0x900008)),
               dict(codes=0x600000, amax_out=0x800000),
               # Overlaps: a row apart, codes on x, h on y.
               dict(y=0x100020), dict(codes=0x100000, row_sinv=0x700000),
               dict(residual=0x200000, h=0x400000, y=0x400000), dict(residual=0x200000, h=0x200020),
               dict(rstd=0x300000)):
        assert _norm(L, **kw) == BAD, kw
    for kw in (dict(cols=16385), dict(rows=1 << 31), dict(x=0x100001), dict(dtype=2, x=0x100002), dict(gamma=0x300001),
               dict(gamma_f32=1, gamma=0x300002), dict(y=0x500001), dict(rstd=0x700002),
               dict(residual=0x200001, h=0x400000),
               dict(codes=0x600000, ring=ops.CRing(0x900000, 0x900040, 0x900044, 0x900048, 0x90004C))):
        assert _norm(L, **kw) == UNSUP, kw
    assert _norm(L, rows=0) == ops.FP8_OK  # nothing to do, nothing launched


def _norm_bwd(L, **kw):
    f = dict(dy=0x100000, h=0x200000, dres=None, dtype=0, rows=4, cols=16, rstd=0x300000, gamma=0x400000, gamma_f32=0,
             dx=0x500000, dgamma=None, workspace=None, workspace_bytes=0)
    f.update(kw)
    return L.fp8_rmsnorm_backward(ctypes.byref(ops.CNormBwdArgs(*f.values())), None)


def test_norm_backward_refusals(L):
    assert L.fp8_rmsnorm_backward(None, None) == BAD
    for kw in (dict(dtype=3), dict(rows=-1), dict(cols=0), dict(dy=None), dict(h=None), dict(rstd=None),
               dict(gamma=None), dict(dx=None), dict(dx=0x200000), dict(dx=0x100020), dict(dgamma=0x500000),
               dict(dgamma=0x600000, workspace=0x600000, workspace_bytes=64)):
        assert _norm_bwd(L, **kw) == BAD, kw
    for kw in (dict(cols=16385), dict(rows=1 << 31), dict(dy=0x100001), dict(dtype=2, h=0x200002), dict(rstd=0x300001),
               dict(dgamma=0x600002)):
        assert _norm_bwd(L, **kw) == UNSUP, kw
    assert _norm_bwd(L, rows=0) == ops.FP8_OK


def test_binding_refuses_cpu_tensors():
    import torch
    x, g = torch.zeros(2, 8), torch.ones(8)
    for call in (lambda: ops.rmsnorm(x, g), lambda: ops.rmsnorm_backward(x, x, torch.ones(2), g)):
        with pytest.raises(ValueError):
            call()


def _act_bwd(L, **kw):
    f = dict(dy=0x100000, dtype=0, z=0x200000, u=None, rows=4, cols=16, act=3, fmt=1, ring=_ring(), ring_u=ops.CRing(),
             amax_out=None, amax_out_u=None, dzq=0x400000, duq=None, db=None, dbu=None, workspace=None,
             workspace_bytes=0)
    f.update(kw)
    return L.fp8_act_backward(ctypes.byref(ops.CActBwdArgs(*f.values())), None)


def test_act_backward_refusals(L):
    assert L.fp8_act_backward(None, None) == BAD
    gate = dict(u=0x300000, ring_u=_ring(0xA00000), duq=0x500000)
    for kw in (dict(dtype=3), dict(rows=-1), dict(cols=-1), dict(act=4), dict(act=-1), dict(fmt=2), dict(dy=None),
               dict(z=None), dict(act=0, z=None, **gate), dict(dzq=None), dict(ring=ops.CRing()),
               dict(u=0x300000), dict(u=0x300000, duq=0x500000), dict(ring_u=_ring(0xA00000)), dict(duq=0x500000),
               dict(gate, ring_u=_ring()), dict(dbu=0x600000), dict(gate, dbu=0x600000), dict(dbu=0x600000, db=0x700000),
               dict(amax_out_u=0x700000), dict(dzq=0x100000), dict(gate, duq=0x400010), dict(db=0x100000),
               dict(db=0x600000, workspace=0x600010, workspace_bytes=64)):
        assert _act_bwd(L, **kw) == BAD, kw
    for kw in (dict(cols=(1 << 30) + 1), dict(rows=1 << 31), dict(dy=0x100001), dict(dtype=2, dy=0x100002),
               dict(z=0x200001), dict(gate, u=0x300001), dict(db=0x600002),
               dict(ring=ops.CRing(0x900000, 0x900040, 0x900044, 0x900048, 0x90004C))):
        assert _act_bwd(L, **kw) == UNSUP, kw


def _mm_act(L, **kw):
    f = dict(A=0x100000, B=0x200000, M=128, N=128, K=128, layout=0, sinv_a=0x300000, sinv_a_rows=0, sinv_b=0x310000,
             bias=None, act=1, aux=None, aux_op=0, z=None, out_kind=0, out=0x400000, out_ring=ops.CRing(), out_amax=None)
    f.update(kw)
    return L.fp8_mm_act(ctypes.byref(ops.CMmActArgs(*f.values())), None)


def test_mm_act_refusals(L):
    assert L.fp8_mm_act(None, None) == BAD
    for kw in (dict(M=-1), dict(N=-1), dict(K=-16), dict(layout=1), dict(layout=2), dict(layout=1 << 10), dict(act=4),
               dict(act=-1), dict(aux_op=2), dict(out_kind=3), dict(out_kind=1), dict(out=None), dict(A=None),
               dict(sinv_a=None), dict(sinv_b=None), dict(out_amax=0x500000), dict(z=0x400100), dict(out=0x100000),
               dict(aux=0x500000, z=0x500000), dict(aux=0x500000, out=0x500002),
               dict(out_kind=1, out=0x500000, aux=0x500000, out_ring=_ring())):
        assert _mm_act(L, **kw) == BAD, kw
    for kw in (dict(K=24), dict(A=0x100008), dict(B=0x200001), dict(out=0x400001), dict(aux=0x500001), dict(z=0x500001),
               dict(bias=0x500002), dict(sinv_a=0x300002),
               dict(out_kind=1, out_ring=ops.CRing(0x900000, 0x900040, 0x900044, 0x900048, 0x90004C))):
        assert _mm_act(L, **kw) == UNSUP, kw
    assert _mm_act(L, M=0) == ops.FP8_OK


def test_packed_arguments_are_the_structures():
    """The bindings pass packed bytes: every field at its structure's offset."""
    for cls, pack in ((ops.CNormArgs, ops._pack_norm), (ops.CNormBwdArgs, ops._pack_norm_bwd),
                      (ops.CMmActArgs, ops._pack_mm_act), (ops.CActBwdArgs, ops._pack_act_bwd)):
        flat = [f for n, f in cls._fields_ for f in ([ctypes.c_void_p] * 5 if f is ops.CRing else [f])]
        raw = pack(*range(1, len(flat) + 1))
        assert len(raw) <= ctypes.sizeof(cls)
        got = cls.from_buffer_copy(raw + b"\0" * (ctypes.sizeof(cls) - len(raw)))
        values = []
        for name, f in cls._fields_:
            v = getattr(got, name)
            values += [getattr(v, n) for n, _ in ops.CRing._fields_] if f is ops.CRing else [v]
        assert values == list(range(1, len(flat) + 1)), cls.__name__


def test_act_backward_refuses_one_amax_for_both_outputs(L):
    gate = dict(u=0x300000, ring_u=_ring(0xA00000), duq=0x500000)
    assert _act_bwd(L, amax_out=0x700000, amax_out_u=0x700000, **gate) == BAD
