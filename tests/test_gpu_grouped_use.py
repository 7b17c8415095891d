"""The grouped products and checkpoints as a program uses them together: a training pass against
64 bits, on another stream, captured and replayed, beside each other; the training example."""
import os
import sys

import pytest
import torch

import grouped_ref as ref
from routed_expert_ffn_top_gb300 import moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import grouped_experts as ex

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def layer(M, H, I, E, k, dtype, seed, drop=0.0):
    g = gen(seed)

    def n(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)
    ids = torch.randn((M, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    if drop:
        ids[torch.rand((M, k), generator=g, device="cuda") < drop] = -1
    w = torch.rand((M, k), generator=g, device="cuda")
    return n(M, H), w, n(E, H, I, std=H ** -0.5), n(E, H, I, std=H ** -0.5), n(E, I, H, std=I ** -0.5), ids, n(M, H)


def through(x, w, wg, wu, wd, ids, d, code):
    """Output and gradients of the example's function."""
    offsets, _, rr = moe.moe_token_plan(ids, wg.shape[0])
    leaves = [t.detach().requires_grad_() for t in (x, w, wg, wu, wd)]
    out = ex.ExpertMLP.apply(*leaves, offsets, rr, code)
    out.backward(d)
    return [out.detach()] + [t.grad for t in leaves]


def exact(x, w, wg, wu, wd, ids, d, code):
    """The same in 64 bits, x, g and u through the checkpoint's codes; code None: not through them."""
    def eight(t):
        if code is None:
            return t
        return ref.values(*ref.quantise(t, code)).to(t.device)
    x, w, wg, wu, wd, d = (t.double() for t in (x, w, wg, wu, wd, d))
    x8 = eight(x)
    out, gx, gw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
    gwg, gwu, gwd = torch.zeros_like(wg), torch.zeros_like(wu), torch.zeros_like(wd)
    for e in range(wg.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        g, u = x[t] @ wg[e], x[t] @ wu[e]
        y = ref.gate(g, u) @ wd[e]
        out.index_add_(0, t, y * w[t, j].unsqueeze(1))
        gw[t, j] = (d[t] * y).sum(1)
        gy = d[t] * w[t, j].unsqueeze(1)
        g, u = eight(g), eight(u)
        gg, gu = ref.gate_grad(gy @ wd[e].t(), g, u).chunk(2, 1)
        gwd[e] = ref.gate(g, u).t() @ gy
        gwg[e], gwu[e] = x8[t].t() @ gg, x8[t].t() @ gu
        gx.index_add_(0, t, gg @ wg[e].t() + gu @ wu[e].t())
    return [out, gx, gw, gwg, gwu, gwd]


# Roundings to the 16-bit type on the longest way (a gradient of x: the gradient of y, of g and u, of the
# rows, the result; out: p, y, the result): at most 4, each at most half a step, 2^-8 or 2^-11, of the
# 2-norm; one more for codes next to a border that fp32 sums put on its other side (one in 10^5 by a step
# of at most 2^-3) and for the sums' own.  Products add no gain beyond the norms': random weights.
BOUND = {BF16: 5 * 2.0 ** -8, F16: 5 * 2.0 ** -11 + 2.0 ** -10}


@pytest.mark.parametrize("M,H,I,E,k,dtype,code,drop", [
    (1, 64, 32, 8, 2, BF16, E4M3, 0.0), (77, 160, 96, 6, 3, BF16, INT8, 0.0), (300, 256, 160, 12, 4, F16, E4M3, 0.1),
    (1000, 352, 224, 5, 2, BF16, E4M3, 0.05), (40, 96, 64, 64, 2, F16, INT8, 0.3), (9, 64, 64, 4, 1, BF16, INT8, 1.0)])
def test_training_pass(M, H, I, E, k, dtype, code, drop):
    args = layer(M, H, I, E, k, dtype, M + H, drop)
    for name, got, want in zip(("out", "x", "weights", "gate", "up", "down"), through(*args, code), exact(*args, code)):
        assert got.shape == want.shape
        assert float((got.double() - want).norm()) <= BOUND[dtype] * float(want.norm()), name


@pytest.mark.parametrize("code,bound", [(E4M3, 0.15), (INT8, 0.06)])
def test_gradients_with_checkpoints_are_near_those_without(code, bound):
    """E4M3 moves a value by at most 2^-4 of itself: x, g and u by 0.063 of the 2-norm each at most, and the
    gate's slope with g, so 0.19 together if all pulled one way; independent roundings add up to about 0.063.
    int8 moves a value by at most the block's largest over 127, some 2.5 to 3 times the block's root mean
    square for normal values: 0.024 each at most, 0.014 in the root mean square."""
    args = layer(500, 256, 160, 6, 2, BF16, 5)
    for got, want in zip(through(*args, code)[1:], exact(*args, None)[1:]):
        assert float((got.double() - want).norm()) <= bound * float(want.norm())


def test_gradient_against_differences():
    """The gradient of x along a direction, from the function's own values: the loss is linear in the
    output, so two outputs a step apart give it up to the curvature and their roundings."""
    x, w, wg, wu, wd, ids, d = layer(400, 128, 96, 4, 2, F16, 6)
    g = through(x, w, wg, wu, wd, ids, d, INT8)[1]
    v = torch.randn(x.shape, generator=gen(7), device="cuda")
    step = 2.0 ** -5
    outs = [exact((x.double() + s * step * v), w, wg, wu, wd, ids, d, None)[0] for s in (1, -1)]
    slope = float(((outs[0] - outs[1]) * d.double()).sum()) / (2 * step)
    got = float((g.double() * v.double()).sum())
    # the gradient's rounding to 8 bits (0.06 of its norm at most, along one direction of 51200), the
    # curvature's share step^2
    assert abs(got - slope) <= 0.06 * float(g.double().norm()) + 2.0 ** -9 * abs(slope)


def test_repeats_bit_for_bit():
    args = layer(700, 256, 192, 16, 4, BF16, 8, 0.1)
    first = through(*args, E4M3)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, through(*args, E4M3)))


def calls(s, stream=None, out=None):
    """One of each call on the tensors of `s`."""
    kw = {"workspace": s["work"], "stream": stream}
    o = out if out is not None else {}
    p, codes, scales = moe.moe_grouped_gated_product(s["rows"], s["wg"], s["wu"], s["off"], checkpoint=E4M3, out=o.get("p"),
                                                     codes=o.get("codes"), scales=o.get("scales"), **kw)
    y = moe.moe_grouped_product(p, s["wd"], s["off"], out=o.get("y"), **kw)
    ggu, again = moe.moe_grouped_gated_product_grad(s["gy"], s["wd"], s["off"], codes, scales, grad_gate_up=o.get("ggu"),
                                                    p=o.get("again"), **kw)
    dx = moe.moe_grouped_product(ggu, (s["wg"], s["wu"]), s["off"], transposed=True, out=o.get("dx"), **kw)
    gw = moe.moe_grouped_weight_grad(s["rows"], ggu, s["off"], out=o.get("gw"), **kw)
    c8, s8 = moe.moe_checkpoint_quantize(s["x"], dtype=INT8, codes=o.get("c8"), scales=o.get("s8"), stream=stream)
    x8 = moe.moe_checkpoint_dequantize(c8, s8, route_row=s["rr"], out=o.get("x8"), stream=stream)
    return {"p": p, "codes": codes, "scales": scales, "y": y, "ggu": ggu, "again": again, "dx": dx, "gw": gw, "c8": c8, "s8": s8, "x8": x8}


def state(seed, M=200, H=128, I=96, E=6, k=3):
    x, _, wg, wu, wd, ids, d = layer(M, H, I, E, k, BF16, seed, 0.1)
    off, _, rr = moe.moe_token_plan(ids, E)
    return {"x": x, "wg": wg, "wu": wu, "wd": wd, "off": off, "rr": rr, "rows": moe.moe_token_sort(x, rr),
            "gy": moe.moe_token_sort(d, rr), "work": torch.zeros(256, dtype=torch.uint8, device="cuda")}


def raw(t):
    return t.view(torch.uint8)


def equal(a, b):
    return [k for k in a if not torch.equal(raw(a[k].contiguous()), raw(b[k].contiguous()))]


def test_another_stream():
    """On a stream of their own, given as an object and as a handle, inputs made on it."""
    want = calls(state(20))
    torch.cuda.synchronize()
    for given in (lambda s: s, lambda s: s.cuda_stream):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            s = state(20)
        got = calls(s, stream=given(side))
        side.synchronize()
        assert equal(got, want) == []
        with torch.cuda.stream(side):
            got = calls(s)
        side.synchronize()
        assert equal(got, want) == []


def test_captured_and_replayed():
    """Replays follow the inputs, the groups' sizes among them; two graphs share a workspace, whose
    status word they only ever set bits of."""
    s, t = state(30), state(31)
    graphs = []
    for q in (s, t):
        q["work"] = s["work"]
        out = {k: torch.empty_like(v) for k, v in calls(q).items()}
        graphs.append((moe.capture_graph(lambda stream, q=q, out=out: calls(q, stream=stream, out=out)), q, out))
    for seed in (32, 33):
        for i, (_, q, _) in enumerate(graphs):
            for k, v in state(seed + 10 * i).items():
                if k != "work":
                    q[k].copy_(v)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for (g, _, out), side in zip(graphs, streams):  # at once
            for v in out.values():
                raw(v).fill_(255)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for i, (_, q, out) in enumerate(graphs):
            assert equal(out, calls(state(seed + 10 * i))) == []
    assert moe.moe_read_device_status(s["work"]) == 0


def test_at_once_on_two_streams():
    want = [calls(state(40 + i, M=900)) for i in range(2)]
    s = [state(40 + i, M=900) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for q, side in zip(s, streams):
            with torch.cuda.stream(side):
                got.append(calls(q))
        torch.cuda.synchronize()
        assert equal(got[0], want[0]) == [] and equal(got[1], want[1]) == []


def test_offsets_that_no_plan_gives():
    """Running backwards, negative and past the rows: clamped, nothing outside is read or written.  (What
    the groups then are is not said; that the call ends and the neighbours stay is.)"""
    g = gen(50)
    rows, w = torch.randn((300, 64), generator=g, device="cuda").to(BF16), torch.randn((4, 64, 64), generator=g, device="cuda").to(BF16)
    for off in ([0, 500, 20, 1 << 30, 300], [-5, -3, 40, 30, 300], [0, 0, 0, 0, (1 << 31) - 1], [300, 200, 100, 0, -1]):
        off = torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
        work = torch.zeros(256, dtype=torch.uint8, device="cuda")
        buf = torch.full((500, 64), 7.0, dtype=BF16, device="cuda")
        moe.moe_grouped_product(rows, w, off, out=buf[100:400], workspace=work)
        moe.moe_grouped_gated_product(rows, w, w, off, checkpoint=E4M3, workspace=work)
        moe.moe_grouped_weight_grad(rows, rows, off, workspace=work)
        assert moe.moe_read_device_status(work) == 0
        assert (buf[:100] == 7.0).all() and (buf[400:] == 7.0).all()


def test_rows_past_four_gigabytes():
    """Byte offsets of rows and results that pass 32 bits, at the ends of both."""
    R, K, N = 1 << 22, 64, 1024
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("memory")
    rows = torch.zeros((R, K), dtype=BF16, device="cuda")
    w = torch.randint(-3, 4, (2, K, N), generator=gen(60), device="cuda").to(BF16)
    tail = torch.randint(-3, 4, (300, K), generator=gen(61), device="cuda").to(BF16)
    rows[-300:] = tail
    off = torch.tensor([0, R - 200, R], dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_product(rows, w, off, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert torch.equal(y[-200:].double(), (tail[100:].double() @ w[1].double()).to(BF16).double())
    assert torch.equal(y[-300:-200].double(), (tail[:100].double() @ w[0].double()).to(BF16).double())
    assert not y[:-300].any()
    c, s = moe.moe_checkpoint_quantize(y, dtype=INT8)
    back = moe.moe_checkpoint_dequantize(c, s)
    assert torch.equal(back[-300:], moe.moe_checkpoint_dequantize(c[-300:].clone(), s[-300:].clone())) and not back[:-300].any()


def test_training_runs():
    for code in (E4M3, INT8):
        losses = ex.train(M=256, H=64, I=96, E=4, k=2, steps=5, code=code)
        assert len(losses) == 5 and all(torch.isfinite(torch.tensor(losses)))

