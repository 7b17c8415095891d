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


def check_plan(ids, E):
    """Against a stable sort: rows, routes and offsets of a plan."""
    offsets, row_route, route_row = moe.moe_token_plan(ids, E)
    flat = ids.reshape(-1)
    R = flat.numel()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, E)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key.long(), minlength=E + 1)
    want = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    want[1:] = counts[:E].cumsum(0)
    assert torch.equal(offsets.long(), want)
    assert torch.equal(row_route.long(), torch.where(valid[order], order, -1))
    rows = torch.empty(R, dtype=torch.int64, device=ids.device)
    rows[order] = torch.arange(R, device=ids.device)
    assert torch.equal(route_row.reshape(-1).long(), torch.where(valid, rows, -1 - rows))


# up to 262,144 routes eight clusters write a plan, past that one more per 4 steps of a run
@pytest.mark.parametrize("M,k,E,drop", [(32768, 8, 128, 0.0), (262145, 1, 128, 0.02), (37500, 8, 128, 0.02), (100003, 3, 7, 0.1),
                                        (131072, 8, 1024, 0.0), (262144, 8, 64, 0.01), (524288, 8, 128, 0.01)])
def test_plan_of_many_routes(M, k, E, drop):
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    if drop:
        bad = torch.rand((M, k), generator=g, device="cuda") < drop
        ids[bad] = torch.where(torch.rand((M, k), generator=g, device="cuda")[bad] < 0.5, -1, E).to(torch.int32)
    check_plan(ids, E)
