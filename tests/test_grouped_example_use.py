"""The grouped-experts example's calls on the CPU, over plain forms of them in 64 bits: what it hands
to them, and what it asks for."""
import pytest
import torch

from test_grouped_example import ex, leaves, plain  # noqa: F401


@pytest.fixture
def calls(plain, monkeypatch):
    """(name, keyword arguments) of the calls made."""
    made = []
    for name in [n for n in vars(ex.moe) if n.startswith(("moe_token_", "moe_grouped_", "moe_checkpoint_"))]:
        def call(*a, real=getattr(ex.moe, name), name=name, **kw):
            made.append((name, kw))
            return real(*a, **kw)
        monkeypatch.setattr(ex.moe, name, call)
    return made


@pytest.mark.parametrize("given", [False, True])
def test_a_status_word_that_nobody_reads_is_not_made(calls, given):
    """Without the caller's status word the calls get none, so each raises what the device found."""
    args, offsets, rr = leaves()
    work = torch.zeros(256, dtype=torch.uint8) if given else None
    ex.ExpertMLP.apply(*args, offsets, rr, None, work).sum().backward()
    grouped = [kw for name, kw in calls if name.startswith("moe_grouped_")]
    assert len(grouped) == 7 and all(kw["workspace"] is work for kw in grouped)


@pytest.mark.parametrize("asked", [(0, 1, 2, 3, 4), (0,), (1,), (2,), (3,), (4,), (0, 1), (2, 3), (1, 4)])
def test_only_the_gradients_asked_for_are_made(calls, asked):
    """Frozen experts, a frozen router, an input without a gradient: the others' gradients are as with all,
    and no call is made for those."""
    args, offsets, rr = leaves()
    ex.ExpertMLP.apply(*args, offsets, rr, None).square().sum().backward()
    want = [t.grad for t in args]
    calls.clear()
    args = [t.detach().requires_grad_(i in asked) for i, t in enumerate(args)]
    ex.ExpertMLP.apply(*args, offsets, rr, None).square().sum().backward()
    assert all((t.grad is None) == (i not in asked) for i, t in enumerate(args))
    assert all(torch.equal(args[i].grad, want[i]) for i in asked)
    names = [name for name, _ in calls]
    assert names.count("moe_grouped_weight_grad") == sum(i in asked for i in (2, 3, 4))
    assert names.count("moe_grouped_product") == 1 + (0 in asked) and names.count("moe_token_sort_grad") == (0 in asked)
    assert names.count("moe_checkpoint_dequantize") == (2 in asked or 3 in asked)
    assert names.count("moe_grouped_gated_product_grad") == (asked != (1,))
