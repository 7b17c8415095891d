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
