"""4-bit block floating point: quantisation bit for bit, products where every sum is exact in
fp32, and the expert step, against plain fp64 forms.

Where scales span only a few powers of two, every partial sum of a product is a multiple of a
power of two below 2^24 times it, so fp32 accumulation in any order is exact and results must
be equal.  Elsewhere a K-long fp32 accumulation errs by at most K 2^-23 sum|terms| (each
addition at most one unit in the last place of fp32).
"""
import pytest
import torch

import tokens_ref as ref
from routed_expert_ffn_top_gb300 import moe, synthetic as syn

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def edge_rows(cols, dtype):
    """Rows with blocks of zeros, ties, saturation, subnormals, the largest values, infinities
    and NaN."""
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]).repeat(4)
    blocks = [torch.zeros(32), ties, -ties, ties * 2.0 ** 10, torch.full((32,), 7.9), torch.full((32,), big),
              torch.full((32,), tiny), torch.full((32,), tiny / 8), torch.linspace(-1, 1, 32) * tiny,
              torch.cat((torch.tensor([float("inf")]), torch.ones(31))),
              torch.cat((torch.ones(31), torch.tensor([float("nan")]))), -torch.zeros(32),
              torch.cat((torch.tensor([4.0]), torch.linspace(0, 4, 31)))]
    n = cols // 32
    rows = [torch.cat([blocks[(i + s) % len(blocks)] for i in range(n)]) for s in range(len(blocks))]
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 64, 0), (7, 480, 0), (21, 2048, 0), (5, 544, 3),
                                           (2, 1568, 8), (130, 768, 0)])
def test_quantise_bit_for_bit(rows, cols, pad, dtype):
    g = gen(rows * cols)
    x = torch.cat((torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-8, 8, (rows, 1), generator=g).float()),
                   edge_rows(cols, dtype).float())).to(dtype)
    R = x.shape[0]
    buf = torch.full((R, cols + pad), float("nan"), dtype=dtype, device="cuda")
    xd = buf[:, :cols]
    xd.copy_(x)
    codes, scales = moe.moe_microscale_quantize(xd)
    want_c, want_s = ref.pack(*ref.quantise(x))
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(codes.cpu(), want_c)
    for out in (torch.bfloat16, torch.float16, torch.float32):
        v = moe.moe_microscale_dequantize(codes, scales, dtype=out).cpu()
        w = ref.values(want_c, want_s).to(out)
        assert torch.equal(torch.isnan(v), torch.isnan(w))
        assert torch.equal(v.nan_to_num(0.0, 1e30, -1e30), w.nan_to_num(0.0, 1e30, -1e30))


def test_quantise_every_bf16_value():
    """All 65536 bf16 patterns, each the largest of its block."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).reshape(-1, 1)
    x = torch.cat((x, x.float().mul(0.4).to(torch.bfloat16), torch.zeros((65536, 30), dtype=torch.bfloat16)), 1)
    codes, scales = moe.moe_microscale_quantize(x.cuda())
    want_c, want_s = ref.pack(*ref.quantise(x))
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(codes.cpu(), want_c)


def test_quantise_into_sorted_rows():
    M, k, E, H = 53, 5, 12, 608
    g = gen(1)
    ids = torch.randint(-1, E, (M, k), generator=g, dtype=torch.int32)
    x = torch.randn((M, H), generator=g).to(torch.bfloat16)
    rr = moe.moe_token_plan(ids.cuda(), E)[2]
    got = moe.moe_microscale_quantize(x.cuda(), route_row=rr)
    rows = moe.moe_token_sort(x.cuda(), rr)
    want = moe.moe_microscale_quantize(rows)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def codes_and_scales(shape, g, lo=126, hi=129):
    """Random codes, scale bytes lo..hi: stored form on the CPU."""
    code = torch.randint(0, 16, shape, generator=g, dtype=torch.uint8)
    byte = torch.randint(lo, hi + 1, shape[:-1] + (shape[-1] // 32,), generator=g, dtype=torch.uint8)
    return ref.pack(code, byte)


def groups(sizes):
    return torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32)


# group sizes around the 128-row tile, empty groups, one row each, more tiles than SMs; widths
# inside, at and past both column tiles; K of one block, inside a stage, across stages
PRODUCTS = [([1], 1, 32), ([3, 0, 1], 64, 64), ([0, 0, 5], 65, 96), ([1] * 8, 200, 256), ([127, 128, 129], 192, 288),
            ([300], 193, 512), ([0, 33, 1, 0, 95, 97], 1000, 1184), ([40] * 30, 96, 160), ([700, 5], 40, 768),
            ([257] * 20, 400, 544), ([31, 32, 64, 96], 7, 2048), ([20000], 70, 32)]


@pytest.mark.parametrize("sizes,N,K", PRODUCTS)
def test_product_exact_sums(sizes, N, K):
    g = gen(N * K)
    E, tail = len(sizes), 3
    R = sum(sizes) + tail
    offsets = groups(sizes)
    xc, xs = codes_and_scales((R, K), g)
    wc, ws = codes_and_scales((E, N, K), g)
    want = ref.product(ref.values(xc, xs), ref.values(wc, ws), offsets)
    args = [t.cuda() for t in (xc, xs, wc, ws)]
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y = moe.moe_microscale_product(*args, offsets=offsets.cuda(), dtype=torch.float32, workspace=work)
    assert moe.moe_read_device_status(work) == 0
    assert torch.equal(y.cpu().double(), want)
    for dt in (torch.bfloat16, torch.float16):
        got = moe.moe_microscale_product(*args, offsets=offsets.cuda(), dtype=dt, workspace=work)
        assert torch.equal(got.cpu(), y.cpu().to(dt))


@pytest.mark.parametrize("N,pad", [(64, 1), (33, 0), (100, 4), (384, 8)])
def test_product_into_strided_rows(N, pad):
    g = gen(N)
    R, K = 150, 128
    xc, xs = codes_and_scales((R, K), g)
    wc, ws = codes_and_scales((1, N, K), g)
    buf = torch.full((R, N + pad), 9.0, device="cuda")
    moe.moe_microscale_product(xc.cuda(), xs.cuda(), wc[0].cuda(), ws[0].cuda(), out=buf[:, :N])
    assert torch.equal(buf[:, :N].cpu().double(), ref.product(ref.values(xc, xs), ref.values(wc, ws), groups([R])))
    assert bool((buf[:, N:] == 9.0).all())


def test_product_scale_range_and_nan():
    """Scales over the whole byte range in their own rows; a NaN block makes its row of x and
    its channel of w NaN and nothing else."""
    g = gen(77)
    R, N, K = 140, 96, 160
    code = torch.randint(0, 16, (R, K), generator=g, dtype=torch.uint8)
    byte = torch.arange(R, dtype=torch.uint8).add(60).unsqueeze(1).expand(R, K // 32).clone()
    byte[5, 2] = 255
    byte[131, 4] = 255
    wcode = torch.randint(0, 16, (1, N, K), generator=g, dtype=torch.uint8)
    wbyte = torch.full((1, N, K // 32), 127, dtype=torch.uint8)
    wbyte[0, 7, 0] = 255
    xc, xs = ref.pack(code, byte)
    wc, ws = ref.pack(wcode, wbyte)
    got = moe.moe_microscale_product(xc.cuda(), xs.cuda(), wc.cuda(), ws.cuda(), dtype=torch.float32).cpu().double()
    nan = torch.zeros((R, N), dtype=torch.bool)
    nan[5], nan[131], nan[:, 7] = True, True, True
    assert torch.equal(torch.isnan(got), nan)
    xv, wv = ref.values(xc, xs).nan_to_num(0.0), ref.values(wc, ws).nan_to_num(0.0)
    want = ref.product(xv, wv, groups([R]))
    assert torch.equal(got[~nan], want[~nan])


def test_product_accumulation_bound_and_invariance():
    """Gaussian data quantised: the accumulation bound, and a row's bits whatever its group,
    its place in the tile and the column tile that the number of rows selects."""
    g = gen(5)
    E, N, K = 4, 256, 2048
    sizes = [150, 1, 200, 33]
    R = sum(sizes)
    xc, xs = moe.moe_microscale_quantize(torch.randn((R, K), generator=g).to(torch.bfloat16).cuda())
    wc, ws = moe.moe_microscale_quantize((torch.randn((E * N, K), generator=g) * 0.02).to(torch.bfloat16).cuda())
    wc, ws = wc.view(E, N, -1), ws.view(E, N, -1)
    offsets = groups(sizes)
    y = moe.moe_microscale_product(xc, xs, wc, ws, offsets=offsets.cuda(), dtype=torch.float32)
    xv, wv = ref.values(xc.cpu(), xs.cpu()), ref.values(wc.cpu(), ws.cpu())
    want = ref.product(xv, wv, offsets)
    bound = K * 2.0 ** -23 * ref.product(xv.abs(), wv.abs(), offsets)
    assert bool(((y.cpu().double() - want).abs() <= bound).all())
    assert float((y.cpu().double() - want).norm() / want.norm()) <= 1e-5
    again = moe.moe_microscale_product(xc, xs, wc, ws, offsets=offsets.cuda(), dtype=torch.float32)
    assert torch.equal(y, again)
    for r in (0, 149, 150, 151, 383):
        e = sum(r >= int(o) for o in offsets[1:])
        one = moe.moe_microscale_product(xc[r:r + 1].contiguous(), xs[r:r + 1].contiguous(), wc[e].contiguous(),
                                         ws[e].contiguous(), dtype=torch.float32)
        assert torch.equal(one[0], y[r])


@pytest.mark.parametrize("sizes,I,K", [([1], 32, 32), ([1] * 8, 96, 256), ([130, 0, 5], 160, 96), ([257, 90], 768, 544),
                                       ([64] * 9, 224, 64), ([500], 544, 128)])
def test_gated_product(sizes, I, K):
    """g and u are exact sums; SiLU(g) u is then within 2^-20 (1 + |g| / 4) of its value (the
    kernel's 2^-21 (1 + |g| / 4), doubled), so its code lies between the codes of the two ends
    of that interval."""
    g = gen(I * K)
    E = len(sizes)
    R = sum(sizes) + 2
    offsets = groups(sizes)
    xc, xs = codes_and_scales((R, K), g, 122, 124)
    wc, ws = codes_and_scales((E, 2 * I, K), g, 126, 127)
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pc, ps = moe.moe_microscale_gated_product(*[t.cuda() for t in (xc, xs, wc, ws)], offsets=offsets.cuda(), workspace=work)
    assert moe.moe_read_device_status(work) == 0
    y = ref.product(ref.values(xc, xs), ref.values(wc, ws), offsets)
    gate, up = y[:, :I], y[:, I:]
    p = gate / (1 + torch.exp(-gate)) * up
    d = 2.0 ** -20 * (1 + gate.abs() / 4)
    lo_c, lo_s = ref.pack(*ref.quantise(p * (1 - d)))
    hi_c, hi_s = ref.pack(*ref.quantise(p * (1 + d)))
    same = lo_s == hi_s
    assert torch.equal(ps.cpu()[same], lo_s[same]) and float(same.double().mean()) > 0.99
    ok = same[:, :I // 32].repeat_interleave(32, 1)
    got = ref.values(pc.cpu(), ps.cpu())
    a, b = ref.values(lo_c, lo_s), ref.values(hi_c, hi_s)
    assert bool(((got >= torch.minimum(a, b)) & (got <= torch.maximum(a, b)))[ok].all())
    assert int(pc[-2:].sum()) == 0 and int(ps[-2:].sum()) == 0


@pytest.mark.parametrize("M,k,E,H,I,drop", [(1, 8, 16, 512, 256, 0), (3, 2, 8, 96, 32, 0.3), (21, 8, 32, 544, 160, 0),
                                            (300, 4, 8, 256, 96, 0.05)])
def test_expert_step(M, k, E, H, I, drop):
    """Rounding y and the sum to bf16 moves each by at most 2^-8 of it, under 2^-9 in the
    2-norm; a p within rounding of a code boundary moves by one code (about one value in 2^18)."""
    g = gen(M * H)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    if drop:
        ids[torch.rand((M, k), generator=g) < drop] = -1
        ids[M // 2] = -1
    w = torch.rand((M, k), generator=g)
    h = torch.randn((M, H), generator=g).to(torch.bfloat16)
    res = torch.randn((M, H), generator=g).to(torch.bfloat16)
    layer = {"H": H, "I": I, "E": E,
             "w_gate": (torch.randn((E, H, I), generator=g) * 0.1).to(torch.bfloat16).cuda(),
             "w_up": (torch.randn((E, H, I), generator=g) * 0.1).to(torch.bfloat16).cuda(),
             "w_down": (torch.randn((E, I, H), generator=g) * 0.1).to(torch.bfloat16).cuda()}
    q = moe.microscale_layer(layer)
    work = moe.microscale_workspace(q, M, k)
    out = moe.moe_microscale_ffn(h.cuda(), q, ids.cuda(), w.cuda(), residual=res.cuda(), workspace=work)
    assert moe.moe_read_device_status(work) == 0
    wq = {n: ref.values(q[n + "_codes"].cpu(), q[n + "_scales"].cpu()) for n in ("gate_up", "down")}
    dense = torch.cat((layer["w_gate"].transpose(1, 2), layer["w_up"].transpose(1, 2)), 1).cpu()
    assert torch.equal(wq["gate_up"], ref.values(*ref.pack(*ref.quantise(dense))))
    x = ref.values(*ref.pack(*ref.quantise(h)))
    want, mag = res.double().clone(), res.double().abs()
    for m in range(M):
        for j in range(k):
            e = int(ids[m, j])
            if not 0 <= e < E:
                continue
            y = wq["gate_up"][e] @ x[m]
            p = y[:I] / (1 + torch.exp(-y[:I])) * y[I:]
            y = wq["down"][e] @ ref.values(*ref.pack(*ref.quantise(p.unsqueeze(0))))[0]
            want[m] += float(w[m, j]) * y
            mag[m] += (float(w[m, j]) * y).abs()
    err = (out.cpu().double() - want).norm()
    assert float(err) <= 2.0 ** -9 * float(mag.norm() + want.norm()) + 1e-3 * float(mag.norm())
    if drop:
        assert torch.equal(out[M // 2].cpu(), res[M // 2])
    again = moe.moe_microscale_ffn(h.cuda(), q, ids.cuda(), w.cuda(), residual=res.cuda(), workspace=work)
    assert torch.equal(out, again)


@pytest.mark.parametrize("M,k,E,H,I,drop", [(1, 8, 128, 2048, 768, 0), (21, 8, 128, 2048, 768, 0), (40, 6, 16, 320, 96, 0.1),
                                            (300, 8, 128, 544, 224, 0.05), (400, 8, 16, 512, 256, 0.02)])
def test_expert_step_is_its_parts(M, k, E, H, I, drop):
    """The step's launches (plan and quantisation in one, at the sizes that take them) give the
    bits of the separate calls; calls share a workspace."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    if drop:
        ids[torch.rand((M, k), generator=g, device="cuda") < drop] = -1
    w = torch.rand((M, k), generator=g, device="cuda")
    h, res = (torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    layer = {"H": H, "I": I, "E": E}
    for name, n, cols in (("gate_up", 2 * I, H), ("down", H, I)):
        c, s = moe.moe_microscale_quantize((torch.randn((E * n, cols), generator=g, device="cuda") * 0.05).to(torch.bfloat16))
        layer[name + "_codes"], layer[name + "_scales"] = c.view(E, n, -1), s.view(E, n, -1)
    offsets, _, rr = moe.moe_token_plan(ids, E)
    x = moe.moe_microscale_quantize(h, route_row=rr)
    p = moe.moe_microscale_gated_product(*x, layer["gate_up_codes"], layer["gate_up_scales"], offsets=offsets)
    y = moe.moe_microscale_product(*p, layer["down_codes"], layer["down_scales"], offsets=offsets)
    want = moe.moe_token_unsort(y, rr, w, residual=res)
    work = moe.microscale_workspace(layer, M, k)
    for _ in range(5):
        out = moe.moe_microscale_ffn(h, layer, ids, w, residual=res, workspace=work)
        assert torch.equal(out, want)
    assert moe.moe_read_device_status(work) == 0


@pytest.mark.parametrize("M,k,E,H,I", [(1, 8, 128, 512, 256), (3, 4, 600, 256, 96), (32, 8, 24, 320, 160),
                                       (33, 8, 24, 320, 160), (256, 1, 16, 512, 256), (700, 4, 40, 512, 256)])
def test_steps_in_a_row_with_routes_of_their_own(M, k, E, H, I):
    """Steps of two layers in a row, each with the rows and routes that the last one's output
    gives and one workspace: the bits of the separate calls, each waited for.  (A step's products
    begin before the kernel ahead has ended: groups or rows of the step before would show.)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(M + k)
    layers = []
    for _ in range(2):
        layer = {"H": H, "I": I, "E": E, "router": torch.randn((H, E), generator=g, device="cuda")}
        for name, n, cols in (("gate_up", 2 * I, H), ("down", H, I)):
            c, s = moe.moe_microscale_quantize((torch.randn((E * n, cols), generator=g, device="cuda") * 0.1).to(torch.bfloat16))
            layer[name + "_codes"], layer[name + "_scales"] = c.view(E, n, -1), s.view(E, n, -1)
        layers.append(layer)
    x0 = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)

    def chain(step):
        x, seen = x0, []
        ids = torch.empty((M, k), dtype=torch.int32, device="cuda")
        for i in range(8):
            layer = layers[i % 2]
            score, idx = torch.topk((x.float() @ layer["router"]) / x.float().norm(dim=1, keepdim=True), k, dim=1)
            ids.copy_(idx)
            if i == 5:
                ids[0, 0] = -1
            x = step(x, layer, ids, torch.softmax(score, dim=1))
            seen.append(x)
            # the step is quadratic in x, so without a norm between the layers eight overflow
            x = torch.nn.functional.rms_norm(x, (H,))
        return torch.stack(seen)

    def parts(x, layer, ids, w):
        offsets, _, rr = moe.moe_token_plan(ids, E)
        q = moe.moe_microscale_quantize(x, route_row=rr)
        torch.cuda.synchronize()
        p = moe.moe_microscale_gated_product(*q, layer["gate_up_codes"], layer["gate_up_scales"], offsets=offsets)
        torch.cuda.synchronize()
        y = moe.moe_microscale_product(*p, layer["down_codes"], layer["down_scales"], offsets=offsets)
        torch.cuda.synchronize()
        return moe.moe_token_unsort(y, rr, w, residual=x)

    work = moe.microscale_workspace(layers[0], M, k)
    want = chain(parts)
    got = chain(lambda x, layer, ids, w: moe.moe_microscale_ffn(x, layer, ids, w, residual=x, workspace=work))
    assert bool(torch.isfinite(want.float()).all())
    assert torch.equal(got, want)
    assert moe.moe_read_device_status(work) == 0


@pytest.mark.parametrize("M,k", [(1, 4), (20, 8), (90, 5)])
def test_steps_in_a_graph(M, k):
    """Three steps captured in a graph on a stream of their own, replayed with other rows and
    routes: the bits of calls outside it."""
    E, H, I = 32, 256, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    layer = {"H": H, "I": I, "E": E}
    for name, n, cols in (("gate_up", 2 * I, H), ("down", H, I)):
        c, s = moe.moe_microscale_quantize((torch.randn((E * n, cols), generator=g, device="cuda") * 0.05).to(torch.bfloat16))
        layer[name + "_codes"], layer[name + "_scales"] = c.view(E, n, -1), s.view(E, n, -1)
    x = torch.zeros((M, H), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((3, M, k), dtype=torch.int32, device="cuda")
    w = torch.full((M, k), 1.0 / k, device="cuda")
    work = moe.microscale_workspace(layer, M, k)

    def steps(ws):
        y = x
        for i in range(3):
            y = moe.moe_microscale_ffn(y, layer, ids[i], w, residual=y, workspace=ws)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps(work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = steps(work)
    other = moe.microscale_workspace(layer, M, k)
    for _ in range(4):
        x.copy_(torch.randn((M, H), generator=g, device="cuda"))
        ids.copy_(torch.randint(-1, E, (3, M, k), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, steps(other))
    assert moe.moe_read_device_status(work) == 0


def test_many_small_gated_units():
    """Many units a CTA with little to do in each: every unit's u is its own."""
    g = gen(11)
    E, I, K = 200, 160, 32
    sizes = [(7 * e) % 33 for e in range(E)]
    R = sum(sizes)
    offsets = groups(sizes).cuda()
    xc, xs = (t.cuda() for t in codes_and_scales((R, K), g, 125, 128))
    wc, ws = (t.cuda() for t in codes_and_scales((E, 2 * I, K), g, 126, 127))
    first = moe.moe_microscale_gated_product(xc, xs, wc, ws, offsets=offsets)
    y = moe.moe_microscale_product(xc, xs, wc, ws, offsets=offsets, dtype=torch.float32)
    gate, up = y[:, :I].double(), y[:, I:].double()
    want = ref.values(*ref.pack(*ref.quantise((gate / (1 + torch.exp(-gate)) * up).cpu())))
    got = ref.values(first[0].cpu(), first[1].cpu())
    assert float(((got - want).abs() > 1e-12).double().mean()) < 1e-4  # values at a code's boundary
    for _ in range(20):
        again = moe.moe_microscale_gated_product(xc, xs, wc, ws, offsets=offsets)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
