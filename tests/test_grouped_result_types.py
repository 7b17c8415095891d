"""The types of results that a caller names and those of the tensors that it gives, on the CPU over a
fake library: a call refuses a pair that does not match."""
import pytest
import torch

from routed_expert_ffn_top_gb300 import moe
from test_grouped_binding import tensors
from test_tokens_binding import fake, launches  # noqa: F401

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = (BF16, F16, F32)


def product(t, **kw):
    return moe.moe_grouped_product(t["rows"], t["gate"], t["off"], workspace=t["work"], **kw)


def weight_grad(t, **kw):
    return moe.moe_grouped_weight_grad(t["rows"], t["p"], t["off"], workspace=t["work"], **kw)


def dequantize(t, **kw):
    return moe.moe_checkpoint_dequantize(t["codes"], t["scales"], **kw)


# call, its result's shape, its type where none is named
CALLS = [(product, (6, 32), BF16), (weight_grad, (3, 64, 32), F32), (dequantize, (6, 64), BF16)]


@pytest.mark.parametrize("call,shape,default", CALLS)
def test_named_given_or_neither(fake, call, shape, default):
    t = tensors()
    assert call(t).dtype is default
    for dtype in TYPES:
        out = torch.zeros(shape, dtype=dtype)
        assert call(t, dtype=dtype).dtype is dtype
        assert call(t, out=out) is out
        assert call(t, out=out, dtype=dtype) is out


@pytest.mark.parametrize("call,shape,default", CALLS)
def test_a_result_of_another_type_than_named_is_refused(fake, call, shape, default):
    t = tensors()
    for dtype in TYPES:
        for given in TYPES:
            if given is not dtype:
                with pytest.raises(TypeError):
                    call(t, dtype=dtype, out=torch.zeros(shape, dtype=given))
    assert launches(fake) == []
