"""The sorted-experts example's autograd functions on the CPU, over plain forms of the calls."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import sorted_experts as ex


@pytest.fixture
def plain(monkeypatch):
    """The four calls in torch for routes that are all valid."""
    def sort(x, rr):
        rows = torch.empty((rr.numel(), x.shape[1]), dtype=x.dtype)
        rows[rr.reshape(-1).long()] = x.repeat_interleave(rr.shape[1], 0)
        return rows
    monkeypatch.setattr(ex.moe, "moe_token_sort", sort)
    monkeypatch.setattr(ex.moe, "moe_token_sort_grad", lambda g, rr: g[rr.long()].sum(1))
    monkeypatch.setattr(ex.moe, "moe_token_unsort", lambda rows, rr, w: (rows[rr.long()] * w.unsqueeze(-1)).sum(1))
    monkeypatch.setattr(ex.moe, "moe_token_unsort_grad", lambda g, rows, rr, w: (
        sort(g, rr) * torch.empty(rr.numel(), 1, dtype=g.dtype).index_copy_(0, rr.reshape(-1).long(), w.reshape(-1, 1)),
        (rows[rr.long()] * g.unsqueeze(1)).sum(-1)))


def test_first_derivatives_match_differences(plain):
    torch.manual_seed(0)
    rr = torch.randperm(12).reshape(4, 3).to(torch.int32)
    x = torch.randn(4, 5, dtype=torch.float64, requires_grad=True)
    rows = torch.randn(12, 5, dtype=torch.float64, requires_grad=True)
    w = torch.randn(4, 3, dtype=torch.float64, requires_grad=True)
    assert torch.autograd.gradcheck(lambda x: ex.SortTokens.apply(x, rr), (x,))
    assert torch.autograd.gradcheck(lambda r, w: ex.UnsortTokens.apply(r, rr, w), (rows, w))


def test_second_derivatives_are_refused(plain):
    """The gradient calls have no derivative of their own: a second one would lack their terms."""
    rr = torch.arange(6, dtype=torch.int32).reshape(2, 3)
    x = torch.ones(2, 4, requires_grad=True)
    (g,) = torch.autograd.grad((ex.SortTokens.apply(x, rr) ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    rows, w = torch.ones(6, 4, requires_grad=True), torch.ones(2, 3, requires_grad=True)
    g, gw = torch.autograd.grad((ex.UnsortTokens.apply(rows, rr, w) ** 2).sum(), (rows, w), create_graph=True)
    with pytest.raises(RuntimeError):
        (g.sum() + gw.sum()).backward()
