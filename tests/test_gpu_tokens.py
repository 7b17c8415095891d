"""Tokens sorted by expert and back, with gradients, against plain fp64 forms.

Bounds.  A sum of n fp32 terms t_i errs by at most n 2^-24 sum|t_i| (first order; doubled
here), and storing a value rounds it by at most u|v| with u = 2^-8 (bf16, 8 significant
bits), 2^-11 (fp16) or 2^-24 (fp32); fp16's smallest step 2^-24 is added below its normal range.
"""
import numpy as np
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


def make_ids(M, k, E, drop, seed):
    g = gen(seed)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    if drop:
        bad = torch.rand((M, k), generator=g) < drop
        ids[bad] = torch.where(torch.rand(int(bad.sum()), generator=g) < 0.5, -1, E).to(torch.int32)
        if M:
            ids[M // 2] = -(2 ** 31)  # a token without any route
    return ids


def check(got, want, bound):
    d = (got.cpu().double() - want).abs()
    assert bool((d <= bound).all()), (float((d - bound).max()), float(d.max()))


def stored(v, dtype):
    return U[dtype] * v.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


# sizes that end inside a warp's step, a warp's run, a CTA and a cluster; one expert, an expert
# count that is no multiple of anything, and the largest
PLANS = [(0, 3, 8, 0), (1, 1, 1, 0), (1, 8, 128, 0), (3, 5, 7, 0.3), (21, 8, 128, 0), (33, 4, 512, 0.1),
         (130, 1, 3, 0), (517, 8, 130, 0.05), (1024, 8, 64, 0), (2049, 16, 1024, 0.02), (5000, 32, 40, 0),
         (20000, 8, 128, 0.01), (70001, 3, 1, 0.5), (64, 2, 16, 1.0)]


@pytest.mark.parametrize("M,k,E,drop", PLANS)
def test_plan_is_the_stable_order(M, k, E, drop):
    ids = make_ids(M, k, E, drop, seed=M + k)
    want = ref.plan(ids, E)
    got = moe.moe_token_plan(ids.cuda(), E)
    again = moe.moe_token_plan(ids.cuda(), E)
    for g, a, w in zip(got, again, want):
        assert torch.equal(g.cpu(), w)
        assert torch.equal(g, a)


def test_plan_of_equal_ids_is_the_identity():
    ids = torch.full((4096, 8), 5, dtype=torch.int32, device="cuda")
    offsets, row_route, route_row = moe.moe_token_plan(ids, 16)
    n = torch.arange(4096 * 8, dtype=torch.int32, device="cuda")
    assert torch.equal(row_route, n) and torch.equal(route_row.reshape(-1), n)
    assert offsets.tolist() == [0] * 6 + [4096 * 8] * 11


def strided(t, pad):
    """The same matrix on the GPU with a longer row pitch (NaN between the rows) and a base
    address off by the padding."""
    if pad == 0:
        return t.cuda()
    R, C = t.shape
    buf = torch.full((R * (C + pad) + pad,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[pad:pad + R * (C + pad)].view(R, C + pad)[:, :C]
    v.copy_(t)
    return v


ROWS = [(1, 8, 128, 2048, 0, 0), (5, 3, 8, 1, 0.2, 0), (21, 8, 128, 2048, 0, 0), (64, 2, 16, 255, 0.1, 0),
        (77, 5, 24, 1033, 0.05, 0), (40, 32, 64, 514, 0.05, 2), (33, 9, 16, 8192 + 8, 0, 8), (300, 8, 32, 96, 1.0, 0),
        (19, 6, 8, 640, 0.1, 1), (700, 1, 8, 130, 0, 3), (30, 17, 32, 520, 0.05, 0), (30, 18, 32, 520, 0.05, 8),
        (9, 32, 64, 1024, 0.05, 0), (50, 9, 16, 776, 0, 0), (60, 2, 8, 4096, 0.1, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,k,E,H,drop,pad", ROWS)
def test_there_and_back_with_gradients(M, k, E, H, drop, pad, dtype):
    g = gen(M * H)
    ids = make_ids(M, k, E, drop, seed=H)
    route_row = ref.plan(ids, E)[2]
    at, live = ref.at_rows(route_row)
    token = torch.arange(M).repeat_interleave(k)
    x, res, gout = (torch.randn((M, H), generator=g).to(dtype) for _ in range(3))
    y = torch.randn((M * k, H), generator=g).to(dtype)
    w = torch.randn((M, k), generator=g)
    y[at[~live]] = float("nan")  # what a dropped route's row holds reaches nothing
    rr, xd, rd, gd, yd = route_row.cuda(), strided(x, pad), strided(res, pad), strided(gout, pad), strided(y, pad)
    wd = w.cuda()

    rows = moe.moe_token_sort(xd, rr)
    want = torch.zeros((M * k, H), dtype=dtype)
    want[at[live]] = x[token[live]]
    assert torch.equal(rows.cpu(), want)

    out = moe.moe_token_unsort(yd, rr, wd, residual=rd)
    t = torch.zeros((M * k, H), dtype=torch.float64)
    t[live] = y[at[live]].double() * w.double().reshape(-1, 1)[live]
    ref_out = t.reshape(M, k, H).sum(1) + res.double()
    mag = t.reshape(M, k, H).abs().sum(1) + res.double().abs()
    check(out, ref_out, 2 * (k + 1) * 2.0 ** -24 * mag + stored(ref_out, dtype))

    gx = moe.moe_token_sort_grad(yd, rr)
    t = torch.zeros((M * k, H), dtype=torch.float64)
    t[live] = y[at[live]].double()
    ref_gx = t.reshape(M, k, H).sum(1)
    check(gx, ref_gx, 2 * k * 2.0 ** -24 * t.reshape(M, k, H).abs().sum(1) + stored(ref_gx, dtype))

    grows, gw = moe.moe_token_unsort_grad(gd, yd, rr, wd)
    ref_g = torch.zeros((M * k, H), dtype=torch.float64)
    ref_g[at[live]] = (gout.double()[token] * w.double().reshape(-1, 1))[live]
    check(grows, ref_g, 2.0 ** -23 * ref_g.abs() + stored(ref_g, dtype))
    prod = torch.zeros((M * k, H), dtype=torch.float64)
    prod[live] = (gout.double()[token][live] * y[at[live]].double())
    check(gw, prod.sum(1).reshape(M, k), (2 * H * 2.0 ** -24 * prod.abs().sum(1)).reshape(M, k))

    again = moe.moe_token_unsort_grad(gd, yd, rr, wd)
    assert torch.equal(again[0], grows) and torch.equal(again[1], gw)


def test_gradients_match_differences():
    """The loss <out, c> in fp64 differences of the plain form, per weight and per row entry."""
    M, k, E, H = 6, 3, 4, 16
    ids = make_ids(M, k, E, 0.2, seed=3)
    route_row = ref.plan(ids, E)[2]
    at, live = ref.at_rows(route_row)
    g = gen(9)
    y, c, w = torch.randn((M * k, H), generator=g), torch.randn((M, H), generator=g), torch.randn((M, k), generator=g)

    def loss(y, w):
        t = torch.zeros((M * k, H), dtype=torch.float64)
        t[live] = y.double()[at[live]] * w.double().reshape(-1, 1)[live]
        return float((t.reshape(M, k, H).sum(1) * c.double()).sum())

    grows, gw = moe.moe_token_unsort_grad(c.cuda(), y.cuda(), route_row.cuda(), w.cuda())
    h = 1e-3  # the loss is linear in each argument: differences are exact up to fp64 rounding
    for m, j in [(0, 0), (2, 1), (M // 2, 2), (5, 2)]:
        e = torch.zeros_like(w, dtype=torch.float64)
        e[m, j] = h
        d = (loss(y, w.double() + e) - loss(y, w.double() - e)) / (2 * h)
        assert abs(d - float(gw[m, j])) <= 1e-5 * H
    for r, i in [(0, 0), (7, 3), (M * k - 1, 15), (11, 8)]:
        e = torch.zeros_like(y, dtype=torch.float64)
        e[r, i] = h
        d = (loss(y.double() + e, w) - loss(y.double() - e, w)) / (2 * h)
        assert abs(d - float(grows[r, i])) <= 1e-5


def test_sort_gradient_is_the_transpose_of_sort():
    """<sort(x), r> = <x, sort_grad(r)> with values whose products and sums are exact."""
    M, k, E, H = 37, 4, 8, 72
    route_row = ref.plan(make_ids(M, k, E, 0.1, seed=4), E)[2].cuda()
    g = gen(5)
    x = torch.randint(-8, 9, (M, H), generator=g).float().cuda()
    r = torch.randint(-8, 9, (M * k, H), generator=g).float().cuda()
    a = (moe.moe_token_sort(x, route_row).double() * r.double()).sum()
    b = (x.double() * moe.moe_token_sort_grad(r, route_row).double()).sum()
    assert float(a) == float(b)


def test_weights_and_residual_are_optional_and_infinities_stay_in_place():
    ids = torch.tensor([[0, 1], [1, -1]], dtype=torch.int32, device="cuda")
    rr = moe.moe_token_plan(ids, 2)[2]
    y = torch.ones((4, 8), device="cuda")
    y[0] = float("inf")  # token 0's first row only
    out = moe.moe_token_unsort(y, rr).cpu()
    assert bool(torch.isinf(out[0]).all()) and bool((out[1] == 1).all())
    grows, gw = moe.moe_token_unsort_grad(torch.ones((2, 8), device="cuda"), y, rr)
    assert bool((grows[:3] == 1).all()) and bool((grows[3] == 0).all())
    assert float(gw[0, 1]) == 8 and float(gw[1, 0]) == 8 and float(gw[1, 1]) == 0


def test_calls_follow_their_stream():
    """Inputs written on a side stream, the calls on the same one, nothing on the default."""
    s = torch.cuda.Stream()
    M, k, E, H = 256, 8, 32, 512
    ids = make_ids(M, k, E, 0, seed=1).pin_memory()
    x = torch.randn((M, H), generator=gen(2)).pin_memory()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        idd, xd = ids.to("cuda", non_blocking=True), x.to("cuda", non_blocking=True)
        rr = moe.moe_token_plan(idd, E)[2]
        rows = moe.moe_token_sort(xd, rr)
        back = moe.moe_token_sort_grad(rows, rr)
    s.synchronize()
    want = torch.zeros_like(x)
    for _ in range(k):  # the sum of the slots in order
        want += x
    assert torch.equal(back.cpu(), want)


def test_bad_route_rows_are_skipped():
    """Entries that no plan writes (past the rows) touch nothing."""
    rr = torch.tensor([[0, 99], [2 ** 30, -(2 ** 30)]], dtype=torch.int32, device="cuda")
    x = torch.ones((2, 32), device="cuda")
    rows = torch.full((4, 32), 7.0, device="cuda")
    moe.moe_token_sort(x, rr, rows=rows)
    assert bool((rows[0] == 1).all()) and bool((rows[1:] == 7).all())
    out = moe.moe_token_unsort(rows, rr)
    assert bool((out[0] == 1).all()) and bool((out[1] == 0).all())
    grows = torch.full((4, 32), 7.0, device="cuda")
    _, gw = moe.moe_token_unsort_grad(x, rows, rr, grad_rows=grows)
    assert bool((grows[0] == 1).all()) and bool((grows[1:] == 7).all())
    assert gw.tolist() == [[32.0, 0.0], [0.0, 0.0]]


def test_rows_past_32_bit_offsets():
    """A sorted matrix of more than 2^32 bytes: the last rows land at the end."""
    M, k, E, H = 4100, 32, 8, 16384
    ids = torch.full((M, k), 3, dtype=torch.int32, device="cuda")
    rr = moe.moe_token_plan(ids, E)[2]
    x = torch.arange(M, device="cuda", dtype=torch.float32).remainder(256).to(torch.bfloat16).unsqueeze(1).expand(M, H).contiguous()
    rows = moe.moe_token_sort(x, rr)
    assert rows.numel() * 2 > 2 ** 32
    assert torch.equal(rows[-k:], x[-1:].expand(k, H)) and torch.equal(rows[:k], x[:1].expand(k, H))
    gx = moe.moe_token_sort_grad(rows, rr)
    assert torch.equal(gx, x * k)
