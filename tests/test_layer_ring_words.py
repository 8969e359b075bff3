"""A ring's words and an amax are memory that a call writes: they are refused where they are
not aligned or lie in another argument, on the host, before CUDA is touched."""

import pytest

from fp8_delayed_scaling_02_b200 import build, ops
from test_layer_capi import BAD, UNSUP, _act_bwd, _mm_act, _norm, _ring

AT = 0x900000


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.lib()


def _with(word, addr):
    r = _ring(AT)
    setattr(r, word, addr)
    return r


NORM = dict(codes=0x600000, ring=_ring(AT))
GATE = dict(u=0x300000, ring_u=_ring(0xA00000), duq=0x500000)
OUT8 = dict(out_kind=1, out_ring=_ring(AT))


@pytest.mark.parametrize("word", ["history", "idx", "scale", "scale_inv"])
def test_words_that_are_not_aligned(L, word):
    odd = _with(word, 0x980002)
    assert _norm(L, codes=0x600000, ring=odd) == UNSUP
    assert _act_bwd(L, ring=odd) == UNSUP
    assert _act_bwd(L, **dict(GATE, ring_u=odd, ring=_ring(0xB00000))) == UNSUP
    assert _mm_act(L, out_kind=1, out_ring=odd) == UNSUP


def test_an_amax_that_is_not_aligned(L):
    assert _norm(L, amax_out=0x980002, **NORM) == UNSUP
    assert _act_bwd(L, amax_out=0x980002) == UNSUP
    assert _act_bwd(L, amax_out_u=0x980001, **GATE) == UNSUP
    assert _mm_act(L, out_amax=0x980002, **OUT8) == UNSUP


@pytest.mark.parametrize("word", ["history", "idx", "scale", "scale_inv", "scratch"])
def test_words_inside_another_argument(L, word):
    for tensor in (0x100000, 0x300000, 0x500000, 0x600000):  # x, gamma, y, codes
        assert _norm(L, codes=0x600000, ring=_with(word, tensor + 8)) == BAD, hex(tensor)
    for tensor in (0x100000, 0x200000, 0x400000):  # dy, z, dzq
        assert _act_bwd(L, ring=_with(word, tensor + 8)) == BAD, hex(tensor)
    for tensor in (0x100000, 0x200000, 0x300000, 0x400000, 0x500000):  # and u, duq
        assert _act_bwd(L, **dict(GATE, ring_u=_with(word, tensor + 8), ring=_ring(0xB00000))) == BAD, hex(tensor)
    for tensor in (0x100000, 0x200000, 0x400000):  # A, B, out
        assert _mm_act(L, out_kind=1, out_ring=_with(word, tensor + 8)) == BAD, hex(tensor)
    # A word that the two rings share, and one that holds the amax.
    shared = _with(word, getattr(_ring(0xA00000), word))
    assert _act_bwd(L, **dict(GATE, ring=shared)) == BAD
    at = getattr(_ring(AT), word)
    assert _norm(L, amax_out=at, **NORM) == BAD
    assert _act_bwd(L, amax_out=at) == BAD
    assert _act_bwd(L, amax_out_u=at, **GATE) == BAD  # the other ring's
    assert _mm_act(L, out_amax=at, **OUT8) == BAD


def test_an_amax_inside_another_argument(L):
    for tensor in (0x100000, 0x300000, 0x500000, 0x600000):
        assert _norm(L, amax_out=tensor + 4, **NORM) == BAD
    for tensor in (0x100000, 0x200000, 0x400000):
        assert _act_bwd(L, amax_out=tensor + 4) == BAD
    for tensor in (0x100000, 0x200000, 0x400000, 0x300000, 0x310000):  # and the two factors
        assert _mm_act(L, out_amax=tensor, **OUT8) == BAD
