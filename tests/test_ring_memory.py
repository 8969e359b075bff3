"""A ring whose buffer's memory is exchanged in place: views and addresses follow it."""

import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops

VIEWS = dict(history=0, idx=16, scale=17, scale_inv=18, scratch=20)


@pytest.mark.parametrize("how", ["data", "set_"])
def test_views_and_addresses_follow_the_memory(how):
    r = ops.Ring("cpu", 2.0)
    for name in VIEWS:
        getattr(r, name)
    r.c()
    other = ops.Ring("cpu", 5.0).buf
    if how == "data":
        r.buf.data = other
    else:
        r.buf.set_(other)
    assert r.scale.item() == 5.0 and r.state()[2] == 5.0
    for name, word in VIEWS.items():
        assert getattr(r, name).data_ptr() == r.buf.data_ptr() + 4 * word, name
        assert getattr(r.c(), name) == r.buf.data_ptr() + 4 * word, name
    assert r._addresses[0] == other.data_ptr()
    r.scale.fill_(7.0)
    assert r.state()[2] == 7.0


def test_a_buffer_that_was_handed_out_before():
    """The next kernel's addresses are the new ones, and the views follow them."""
    r = ops.Ring("cpu", 2.0)
    b = r.buf
    for name in VIEWS:
        getattr(r, name)
    old, c = r._addresses, r.c()
    b.data = ops.Ring("cpu", 5.0).buf
    assert r._addresses[0] == b.data_ptr() != old[0]
    assert r.c() is not c and r.c().scale == b.data_ptr() + 17 * 4
    assert r.scale.item() == 5.0


def test_views_are_kept_while_the_memory_stays():
    r = ops.Ring("cpu")
    assert r.scale is r.scale and r.c() is r.c()
