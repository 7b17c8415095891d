"""The grouped-experts example's autograd function on the CPU, over plain forms of the calls in 64
bits whose checkpoints keep their values: its gradients against differences."""
import os
import sys

import pytest
import torch

import grouped_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import grouped_experts as ex


@pytest.fixture
def plain(monkeypatch):
    """The calls in torch for routes that are all valid."""
    def sort(x, rr):
        rows = torch.empty((rr.numel(), x.shape[1]), dtype=x.dtype)
        rows[rr.reshape(-1).long()] = x.repeat_interleave(rr.shape[1], 0)
        return rows

    def gated(rows, wg, wu, off, checkpoint=None, workspace=None):
        g, u = ref.product(rows, wg, off), ref.product(rows, wu, off)
        return ref.gate(g, u), torch.cat((g, u), 1), torch.zeros(1)

    def gated_grad(gy, wd, off, codes, scales, workspace=None):
        g, u = codes.chunk(2, 1)
        return ref.gate_grad(ref.product(gy, wd, off, True), g, u), ref.gate(g, u)

    def product(rows, w, off, transposed=False, workspace=None):
        if isinstance(w, tuple):
            return sum(ref.product(r, m, off, transposed) for r, m in zip(rows.chunk(2, 1), w))
        return ref.product(rows, w, off, transposed)
    for name, f in {
            "moe_token_sort": sort, "moe_token_sort_grad": lambda g, rr: g[rr.long()].sum(1),
            "moe_token_unsort": lambda rows, rr, w: (rows[rr.long()] * w.unsqueeze(-1)).sum(1),
            "moe_token_unsort_grad": lambda g, rows, rr, w: (
                sort(g, rr) * torch.empty(rr.numel(), 1, dtype=g.dtype).index_copy_(0, rr.reshape(-1).long(), w.reshape(-1, 1)),
                (rows[rr.long()] * g.unsqueeze(1)).sum(-1)),
            "moe_grouped_gated_product": gated, "moe_grouped_gated_product_grad": gated_grad, "moe_grouped_product": product,
            "moe_grouped_weight_grad": lambda rows, grads, off, dtype=None, workspace=None: ref.weight_grad(rows, grads, off),
            "moe_checkpoint_quantize": lambda x, dtype=None: (x.clone(), torch.zeros(1)),
            "moe_checkpoint_dequantize": lambda c, s, dtype=None, route_row=None: sort(c, route_row)}.items():
        monkeypatch.setattr(ex.moe, name, f)


def leaves():
    torch.manual_seed(0)
    M, k, H, I, E = 4, 2, 5, 3, 3
    offsets = torch.tensor([0, 3, 3, 8], dtype=torch.int32)  # one expert without rows
    rr = torch.randperm(M * k).reshape(M, k).to(torch.int32)
    shapes = ((M, H), (M, k), (E, H, I), (E, H, I), (E, I, H))
    return [torch.randn(s, dtype=torch.float64, requires_grad=True) for s in shapes], offsets, rr


def test_first_derivatives_match_differences(plain):
    args, offsets, rr = leaves()
    assert torch.autograd.gradcheck(lambda *a: ex.ExpertMLP.apply(*a, offsets, rr, None), args)


def test_second_derivatives_are_refused(plain):
    args, offsets, rr = leaves()
    g = torch.autograd.grad((ex.ExpertMLP.apply(*args, offsets, rr, None) ** 2).sum(), args, create_graph=True)
    with pytest.raises(RuntimeError):
        sum(t.sum() for t in g).backward()


def test_memory_kept():
    a, b = ex.memory()
    assert b < a / 2
