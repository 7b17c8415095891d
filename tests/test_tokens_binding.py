"""What the token and 4-bit calls check before anything is launched, on the CPU: a fake library
records the calls that would have reached the GPU."""
import ctypes

import pytest
import torch

import __graft_entry__ as entry
from routed_expert_ffn_top_gb300 import moe

A = 1 << 20  # an aligned address; never dereferenced by validation


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return moe.lib()


@pytest.mark.parametrize("name", ["gate_up_codes", "gate_up_scales", "down_codes", "down_scales"])
def test_expert_step_refuses_weights_before_a_launch(lib, name):
    """Launching here, without a device, would come back as MOE_ERR_CUDA."""
    for bad in (None, A + 8):
        w = moe.MicroscaleWeights(64, 32, 4, 0, A, A, A, A)
        setattr(w, name, bad)
        for M in (4, 200):  # both forms of the plan
            assert lib.moe_microscale_ffn(A, ctypes.byref(w), M, 2, A, A, None, A, A, 1 << 30, None) == moe.MOE_ERR_INVALID_ARG
