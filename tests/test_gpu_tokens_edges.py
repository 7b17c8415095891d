"""The token sort past the sizes of its forms: rows that one, two or more vectors a thread cover."""
import pytest
import torch

import tokens_ref as ref
from routed_expert_ffn_top_gb300 import moe

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("H", [65, 127, 129, 254, 257, 258, 385, 514, 515])
def test_unsort_gradients_of_narrow_rows(H, dtype):
    """Bounds: a stored value errs by U of it, a sum of H fp32 products by 2 H 2^-24 of their
    magnitudes' sum."""
    M, k, E = 53, 9, 12
    g = gen(H)
    ids = torch.randint(-1, E, (M, k), generator=g, dtype=torch.int32)
    route_row = ref.plan(ids, E)[2]
    at, live = ref.at_rows(route_row)
    token = torch.arange(M).repeat_interleave(k)
    gout, y = torch.randn((M, H), generator=g).to(dtype), torch.randn((M * k, H), generator=g).to(dtype)
    w = torch.randn((M, k), generator=g)
    grows, gw = moe.moe_token_unsort_grad(gout.cuda(), y.cuda(), route_row.cuda(), w.cuda())
    want = torch.zeros((M * k, H), dtype=torch.float64)
    want[at[live]] = (gout.double()[token] * w.double().reshape(-1, 1))[live]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    assert bool(((grows.cpu().double() - want).abs() <= (2.0 ** -23 + U[dtype]) * want.abs() + tiny).all())
    prod = torch.zeros((M * k, H), dtype=torch.float64)
    prod[live] = gout.double()[token][live] * y[at[live]].double()
    bound = 2 * H * 2.0 ** -24 * prod.abs().sum(1)
    assert bool(((gw.cpu().double().reshape(-1) - prod.sum(1)).abs() <= bound).all())
