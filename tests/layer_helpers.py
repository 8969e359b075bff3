"""Shared helpers of the tests of the norm, the activation product and their gradients."""

import numpy as np
import torch

from oracle import fp8_formats as OF

U = 2.0 ** -24  # half a float32 step, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# Half the smallest step: what a rounding to the type costs below its normal range.
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def at_offset(t, offset):
    """A CUDA copy of ``t`` that starts ``offset`` elements past a 256-byte aligned address."""
    flat = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    flat[offset:].copy_(t.reshape(-1))
    return flat[offset:].view(t.shape)


def assert_within(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    tol = np.broadcast_to(np.asarray(tol, np.float64), ref.shape)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(got - ref)[bad] / np.maximum(tol[bad], 1e-300)):.3g} x the tolerance, first at "
                           f"{tuple(int(b[0]) for b in np.nonzero(bad))}")


def assert_codes(codes, v, tol, fmt, what):
    """Every code lies between the codes of the two ends of the interval v +- tol of the
    scaled value: conversion is monotone, so where both ends have one code it is exact."""
    with np.errstate(over="ignore"):
        lo = OF.decode(OF.encode((v - tol).astype(np.float32), fmt), fmt)
        hi = OF.decode(OF.encode((v + tol).astype(np.float32), fmt), fmt)
    got = OF.decode(codes.cpu().numpy(), fmt)
    bad = ~((lo <= got) & (got <= hi))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} codes outside, first at " \
                          f"{tuple(int(b[0]) for b in np.nonzero(bad))}"
    # That the interval is narrow is a statement about many values: among n of them one that
    # cancels to near zero, where E5M2's steps are finer than the sum's own error, is a share
    # of 1/n, so below 256 values the share says nothing about the tolerance.
    if v.size >= 256:
        assert float(np.mean(lo == hi)) > 0.9, f"{what}: the tolerance decides too many codes"


def assert_folded(before, ring, amax, tol, fmt):
    """The ring folded one amax within ``tol`` of ``amax``; the rest follows from its own value."""
    h0, i0, s0, _, _ = before
    h1, i1, s1, si1, scratch = ring.state()
    assert i1 == (i0 + 1) % 16
    a = float(h1[i0])
    assert abs(a - amax) <= tol, (a, amax, tol)
    h0 = h0.clone()
    h0[i0] = a
    assert torch.equal(h0, h1)
    m = np.float32(h1.max())
    fmax = np.float32(448.0 if fmt == OF.E4M3 else 57344.0)
    assert np.float32(s1) == (np.float32(fmax / m) if m > 0 else np.float32(s0))
    assert np.float32(si1) == np.float32(1.0) / np.float32(s0)
    assert all(int(v) == 0 for v in scratch), "scratch must self-reset"
