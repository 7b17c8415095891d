"""Forms of the grouped calls that a program may use beside the usual ones, and what the training
example keeps and reports."""
import pytest
import torch

import grouped_ref as ref
from routed_expert_ffn_top_gb300 import moe
from test_gpu_grouped_use import BOUND, E4M3, F16, INT8, ex, gen, layer

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def workspace():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M,H,I,E,k", [(64, 512, 256, 8, 2), (77, 160, 96, 6, 3)])
def test_memory_kept_is_as_stated(M, H, I, E, k):
    """The bytes that the function keeps for its way back, beside the weights and the plan."""
    x, w, wg, wu, wd, ids, d = layer(M, H, I, E, k, BF16, M)
    offsets, _, rr = moe.moe_token_plan(ids, E)
    leaves = [t.detach().requires_grad_() for t in (x, w, wg, wu, wd)]
    there = {t.data_ptr() for t in (*leaves, offsets, rr)}
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        out = ex.ExpertMLP.apply(*leaves, offsets, rr, INT8, workspace())
    new = {t.data_ptr(): t.numel() * t.element_size() for t in kept if t.data_ptr() not in there}
    assert sum(new.values()) == ex.memory(M, H, I, k)[1]
    out.backward(d)
