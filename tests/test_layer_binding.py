"""The Python calls of the operators around the linear take their arguments as their signatures say."""

import inspect

import pytest
import torch

from fp8_delayed_scaling_02_b200 import ops

CALLS = {
    ops.rmsnorm: dict(x=torch.zeros(2, 16), gamma=torch.ones(16)),
    ops.rmsnorm_backward: dict(dy=torch.zeros(2, 16), h=torch.zeros(2, 16), rstd=torch.ones(2), gamma=torch.ones(16)),
    ops.mm_act: dict(a=torch.zeros(2, 16, dtype=torch.uint8), b=torch.zeros(4, 16, dtype=torch.uint8),
                     sinv_a=torch.ones(1), sinv_b=torch.ones(1)),
    ops.act_backward: dict(dy=torch.zeros(2, 16), z=torch.zeros(2, 16, dtype=torch.bfloat16), act=ops.ACT_SILU,
                           fmt=ops.E5M2, ring=ops.Ring("cpu")),
}


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_every_argument_may_be_a_keyword(call):
    kw = CALLS[call]
    inspect.signature(call).bind(**kw, stream=None)
    names = list(inspect.signature(call).parameters)
    assert names[:len(kw)] == list(kw) and names[-1] == "stream"
    for k in range(len(kw) + 1):  # the first k by position
        by_place, by_name = list(kw.values())[:k], dict(list(kw.items())[k:])
        with pytest.raises(ValueError, match="CUDA tensors"):  # got as far as looking at the tensor
            call(*by_place, **by_name)
    with pytest.raises(TypeError, match=names[0]):
        call()
