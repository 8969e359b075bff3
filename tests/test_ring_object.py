"""The Python object that holds a ring: its views and addresses follow its buffer."""

import copy
import pickle

import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops

VIEWS = ("history", "idx", "scale", "scale_inv", "scratch")


def test_views_made_in_inference_mode_stay_writable():
    r = ops.Ring("cpu", 2.0)
    with torch.inference_mode():
        for name in VIEWS:
            getattr(r, name)
    with torch.no_grad():
        r.idx.fill_(3)
    r.scale.fill_(4.0)
    assert r.state()[1:3] == (3, 4.0)
    assert not any(getattr(r, name).is_inference() for name in VIEWS)


@pytest.mark.parametrize("name", VIEWS)
def test_views_cannot_be_assigned(name):
    r = ops.Ring("cpu")
    with pytest.raises(AttributeError):
        setattr(r, name, torch.zeros(1))
    getattr(r, name)
    with pytest.raises(AttributeError):
        setattr(r, name, torch.zeros(1))


def test_own_attributes_survive_a_new_buffer_and_copies():
    r = ops.Ring("cpu", 2.0)
    r.label = "input"
    old = r.scale, r.c().scale
    r.buf = r.buf.clone()
    assert r.label == "input" and r.scale.item() == 2.0
    assert r.scale.data_ptr() != old[0].data_ptr() and r.c().scale == r.scale.data_ptr() != old[1]
    for d in (copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert d.label == "input" and d.scale.item() == 2.0
        assert d.c().scale == d.scale.data_ptr() == d.buf.data_ptr() + 17 * 4 != r.scale.data_ptr()
        d.scale.fill_(8.0)
        assert r.scale.item() == 2.0
    shallow = copy.copy(r)
    assert shallow.label == "input" and shallow.buf is r.buf
    shallow.buf = shallow.buf.clone()  # the other's views stay with its buffer
    assert r.c().scale == r.scale.data_ptr() == r.buf.data_ptr() + 17 * 4
