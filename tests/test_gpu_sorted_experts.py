"""The sorted-experts example: its gradients against torch's own over the same layer, its
training, and the 4-bit step beside the dense block."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import sorted_experts as ex

pytestmark = pytest.mark.gpu


def test_gradients_match_autograd():
    """fp32 sums of at most 96 + 64 terms a value through three products: 1e-4 of the gradient's
    norm is over 100 times their rounding."""
    torch.manual_seed(1)
    M, H, I, E, k = 37, 48, 64, 6, 3
    layer = ex.SortedExperts(H, I, E, k).cuda()
    x = torch.randn(M, H, device="cuda", requires_grad=True)
    c = torch.randn(M, H, device="cuda")
    (layer(x) * c).sum().backward()
    got = [x.grad] + [p.grad for p in layer.parameters()]

    xd = x.detach().double().requires_grad_()
    ps = [p.detach().double().requires_grad_() for p in layer.parameters()]
    ids, _ = layer.route(x.detach())
    router, gate, up, down = ps
    w = torch.softmax((xd @ router).gather(1, ids.long()), 1)
    h = xd.unsqueeze(1).unsqueeze(2)  # [M,1,1,H]
    y = (torch.nn.functional.silu(h @ gate[ids.long()]) * (h @ up[ids.long()])) @ down[ids.long()]
    ((y.squeeze(2) * w.unsqueeze(2)).sum(1) * c.double()).sum().backward()
    for a, b in zip(got, [xd.grad] + [p.grad for p in ps]):
        assert float((a.double() - b).norm()) <= 1e-4 * float(b.norm())


def test_training_lowers_the_loss():
    losses = ex.train(M=128, H=32, I=48, E=4, k=2, steps=30)
    assert losses[-1] < 0.5 * losses[0]


def test_serving_beside_the_dense_block():
    """Rounding to 4 bits moves a value by up to a sixth of itself, a tenth in the 2-norm; x, p and
    two weights are rounded, so the result differs by a few tenths at most."""
    for M, err, _, _ in ex.serve(H=512, I=256, E=16, k=4, sizes=(1, 5, 130)):
        assert 0.01 < err < 0.4, (M, err)
