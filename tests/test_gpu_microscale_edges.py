"""4-bit products, the expert step and quantisation at the ends of their ranges."""
import pytest
import torch

import tokens_ref as ref
from routed_expert_ffn_top_gb300 import moe

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def test_product_of_rows_past_2_gb():
    """fp32 rows of more than 2^31 bytes: their columns lie past a tensor store's coordinates.
    Channels of zeros but for three windows, whose sums are exact."""
    R, K, N = 33, 32, 2 ** 29 + 1024
    if torch.cuda.mem_get_info()[0] < 110 * 2 ** 30:
        pytest.skip("needs 110 GB of device memory")
    windows = [(0, 256), (2 ** 29 - 128, 2 ** 29 + 128), (N - 256, N)]
    g = gen(1)
    xc = torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8)
    xs = torch.full((R, 16), 127, dtype=torch.uint8)
    wc = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((N, 16), 127, dtype=torch.uint8, device="cuda")
    part = {}
    for lo, hi in windows:
        c = torch.randint(0, 256, (hi - lo, K // 2), generator=g, dtype=torch.uint8)
        wc[lo:hi] = c.cuda()
        part[lo] = ref.values(xc, xs[:, :1]) @ ref.values(c, torch.full((hi - lo, 1), 127, dtype=torch.uint8)).T
    y = torch.full((R, N), float("nan"), device="cuda")
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_microscale_product(xc.cuda(), xs.cuda(), wc, ws, out=y, workspace=work)
    assert moe.moe_read_device_status(work) == 0
    for lo, hi in windows:
        assert torch.equal(y[:, lo:hi].cpu().double(), part[lo])
    for r in (0, R - 1):
        for lo, hi in ((256, 2 ** 29 - 128), (2 ** 29 + 128, N - 256)):
            assert int(torch.count_nonzero(y[r, lo:hi])) == 0  # a NaN counts
    del y, wc, ws
    torch.cuda.empty_cache()


def make_layer(E, H, I, seed, gain=0.05):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    layer = {"H": H, "I": I, "E": E}
    for name, n, cols in (("gate_up", 2 * I, H), ("down", H, I)):
        c, s = moe.moe_microscale_quantize((torch.randn((E * n, cols), generator=g, device="cuda") * gain).to(torch.bfloat16))
        layer[name + "_codes"], layer[name + "_scales"] = c.view(E, n, -1), s.view(E, n, -1)
    return layer


def parts(h, layer, ids, w, residual=None):
    """The expert step by its separate calls, each waited for."""
    offsets, _, rr = moe.moe_token_plan(ids, layer["E"])
    q = moe.moe_microscale_quantize(h, route_row=rr)
    torch.cuda.synchronize()
    p = moe.moe_microscale_gated_product(*q, layer["gate_up_codes"], layer["gate_up_scales"], offsets=offsets)
    torch.cuda.synchronize()
    y = moe.moe_microscale_product(*p, layer["down_codes"], layer["down_scales"], offsets=offsets)
    torch.cuda.synchronize()
    return moe.moe_token_unsort(y, rr, w, residual=residual)


@pytest.mark.parametrize("M,k,I", [(1, 8, 96), (21, 8, 768), (300, 4, 96)])
def test_step_behind_work_longer_than_its_waits(M, k, I):
    """Queued behind work that takes longer than a bounded wait, with units of few stages (a
    CTA's copies then never come round its ring): no wait runs out."""
    E, H = 64, 256
    layer = make_layer(E, H, I, seed=M)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((M, k), generator=g, device="cuda")
    h = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    want = parts(h, layer, ids, w)
    work = moe.microscale_workspace(layer, M, k)
    torch.cuda.synchronize()
    torch.cuda._sleep(3_500_000_000)  # over a second and a half at any SM clock
    out = moe.moe_microscale_ffn(h, layer, ids, w, workspace=work)
    assert moe.moe_read_device_status(work) == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("M,k", [(1, 4), (20, 8), (90, 5)])
def test_replayed_steps_with_other_weights(M, k):
    """Steps in a graph whose route weights change in place, from replay to replay and within
    one: what the way back reads before the kernel ahead has ended is this step's."""
    E, H, I = 32, 256, 128
    layer = make_layer(E, H, I, seed=M)
    g = torch.Generator(device="cuda")
    g.manual_seed(M + 1)
    x = torch.zeros((M, H), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((M, k), dtype=torch.int32, device="cuda")
    scale, w = torch.zeros((4, M, k), device="cuda"), torch.zeros((M, k), device="cuda")

    def steps(ws):
        outs = []
        for i in range(4):
            w.copy_(scale[i])
            outs.append(moe.moe_microscale_ffn(x, layer, ids, w, residual=x, workspace=ws))
        return torch.stack(outs)

    work = moe.microscale_workspace(layer, M, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps(work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = steps(work)
    for _ in range(6):
        x.copy_(torch.randn((M, H), generator=g, device="cuda"))
        ids.copy_(torch.randint(-1, E, (M, k), generator=g, device="cuda"))
        scale.copy_(torch.rand((4, M, k), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = torch.stack([parts(x, layer, ids, scale[i], residual=x) for i in range(4)])
        assert torch.equal(out, want)
    assert moe.moe_read_device_status(work) == 0


def test_calls_on_a_stream_that_is_not_current():
    """Calls given a busy stream, with outputs and workspaces of their own, while the current
    stream allocates and overwrites as much memory right after each."""
    M, k, E, H, I = 300, 4, 16, 512, 256
    layer = make_layer(E, H, I, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((M, k), generator=g, device="cuda")
    h = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    offsets, row_route, rr = moe.moe_token_plan(ids, E)
    rows = moe.moe_token_sort(h, rr)
    q = moe.moe_microscale_quantize(h, route_row=rr)
    p = moe.moe_microscale_gated_product(*q, layer["gate_up_codes"], layer["gate_up_scales"], offsets=offsets)
    y = moe.moe_microscale_product(*p, layer["down_codes"], layer["down_scales"], offsets=offsets)
    dense = {"H": H, "I": I, "E": E}
    for name, n, cols in (("w_gate", H, I), ("w_up", H, I), ("w_down", I, H)):
        dense[name] = torch.randn((E, n, cols), generator=g, device="cuda").to(torch.bfloat16)
    four = moe.microscale_layer(dense)
    calls = [(lambda s: moe.moe_token_plan(ids, E, stream=s), (offsets, row_route, rr)),
             (lambda s: moe.moe_token_sort(h, rr, stream=s), rows),
             (lambda s: moe.moe_token_sort_grad(rows, rr, stream=s), moe.moe_token_sort_grad(rows, rr)),
             (lambda s: moe.moe_token_unsort(y, rr, w, residual=h, stream=s), moe.moe_token_unsort(y, rr, w, residual=h)),
             (lambda s: moe.moe_token_unsort_grad(h, y, rr, w, stream=s), moe.moe_token_unsort_grad(h, y, rr, w)),
             (lambda s: moe.moe_microscale_quantize(h, route_row=rr, stream=s), q),
             (lambda s: moe.moe_microscale_dequantize(*q, stream=s), moe.moe_microscale_dequantize(*q)),
             (lambda s: moe.moe_microscale_gated_product(*q, layer["gate_up_codes"], layer["gate_up_scales"],
                                                         offsets=offsets, stream=s), p),
             (lambda s: moe.moe_microscale_product(*p, layer["down_codes"], layer["down_scales"], offsets=offsets, stream=s), y),
             (lambda s: moe.microscale_layer(dense, stream=s), four),
             (lambda s: moe.moe_microscale_ffn(h, layer, ids, w, residual=h, stream=s),
              moe.moe_microscale_ffn(h, layer, ids, w, residual=h))]

    def tensors(v):
        if isinstance(v, torch.Tensor):
            return [v]
        return [t for t in (v.values() if isinstance(v, dict) else v) if isinstance(t, torch.Tensor)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, 0):
        for call, want in calls:
            torch.cuda.synchronize()
            # this stream's pool holds freed blocks of every size that the call might take
            free = [torch.zeros(t.numel() * t.element_size(), dtype=torch.uint8, device="cuda") for t in tensors(want)]
            free.append(moe.microscale_workspace(layer, M, k))
            sizes = [f.numel() for f in free]
            del free
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
            got = call(stream)
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
            torch.cuda.synchronize()
            for a, b in zip(tensors(got), tensors(want)):
                assert torch.equal(a, b)
            del junk, got


def test_calls_without_a_workspace():
    """They wait for their result and raise what the status word says; in a graph's capture they
    do neither."""
    M, k, E, H, I = 5, 3, 8, 256, 128
    layer = make_layer(E, H, I, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((M, k), generator=g, device="cuda")
    h = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    want = parts(h, layer, ids, w)
    done = torch.cuda.Event()
    torch.cuda._sleep(10_000_000)
    done.record()
    assert torch.equal(moe.moe_microscale_ffn(h, layer, ids, w), want)
    assert done.query()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.moe_microscale_ffn(h, layer, ids, w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    zeros = torch.zeros
    torch.zeros = lambda *a, **kw: zeros(*a, **kw).fill_(moe.MOE_DEV_WAIT_TIMEOUT)  # a word that is set
    try:
        with pytest.raises(moe.MoeError):
            moe.moe_microscale_product(*moe.moe_microscale_quantize(h), layer["gate_up_codes"][0], layer["gate_up_scales"][0])
    finally:
        torch.zeros = zeros


@pytest.mark.parametrize("M,k", [(3, 4), (40, 8), (300, 4)])
def test_step_reads_nothing_that_a_workspace_held(M, k):
    """All but the status word of the workspace holds bytes that are NaN scales, dropped rows and
    far offsets to any reader; some routes are dropped."""
    E, H, I = 16, 320, 96
    layer = make_layer(E, H, I, seed=M)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    ids = torch.randint(-1, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((M, k), generator=g, device="cuda")
    h = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    want = parts(h, layer, ids, w)
    work = moe.microscale_workspace(layer, M, k)
    assert int(work[:256].count_nonzero()) == 0
    for byte in (0, 255):
        work[256:] = byte
        assert torch.equal(moe.moe_microscale_ffn(h, layer, ids, w, workspace=work), want)
    assert moe.moe_read_device_status(work) == 0


def test_status_of_a_workspace_that_only_the_products_take():
    """A 16-byte aligned one: its status word is read back and cleared like any other."""
    x, wt = moe.moe_microscale_quantize(torch.ones((3, 64), device="cuda")), moe.moe_microscale_quantize(torch.ones((5, 64), device="cuda"))
    buf = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    for at in (16, 48, 256):
        work = buf[at:at + 256]
        y = moe.moe_microscale_product(*x, *wt, workspace=work)
        assert bool((y == 64).all())
        assert moe.moe_read_device_status(work) == 0
        work[0] = moe.MOE_DEV_WAIT_TIMEOUT
        assert moe.moe_read_device_status(work) == moe.MOE_DEV_WAIT_TIMEOUT
        assert moe.moe_read_device_status(work) == 0


@pytest.mark.parametrize("M,k,E,H,I,res", [(1, 8, 128, 2048, 768, False), (21, 8, 128, 2048, 768, True), (40, 6, 16, 320, 96, True),
                                           (300, 8, 128, 544, 224, False), (400, 8, 16, 512, 256, True),
                                           (30, 17, 32, 96, 64, True), (30, 18, 32, 96, 64, False), (30, 18, 32, 96, 64, True),
                                           (50, 32, 40, 160, 32, True)])
def test_step_with_unrounded_rows(M, k, E, H, I, res):
    """y_dtype float32: the bits of the separate calls in fp32, rounded once.  The result without
    a residual then errs by the rounding of out alone, 2^-9 of it at most in the 2-norm."""
    layer = make_layer(E, H, I, seed=M)
    g = torch.Generator(device="cuda")
    g.manual_seed(M + k)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    if M > 30:
        ids[torch.rand((M, k), generator=g, device="cuda") < 0.05] = -1
    w = torch.rand((M, k), generator=g, device="cuda")
    h = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16) if res else None
    offsets, _, rr = moe.moe_token_plan(ids, E)
    q = moe.moe_microscale_quantize(h, route_row=rr)
    p = moe.moe_microscale_gated_product(*q, layer["gate_up_codes"], layer["gate_up_scales"], offsets=offsets)
    y = moe.moe_microscale_product(*p, layer["down_codes"], layer["down_scales"], offsets=offsets, dtype=torch.float32)
    want = moe.moe_token_unsort(y, rr, w, residual=r.float() if res else None)
    half = moe.moe_microscale_ffn(h, layer, ids, w, residual=r, workspace=moe.microscale_workspace(layer, M, k))
    layer["y_dtype"] = torch.float32
    work = moe.microscale_workspace(layer, M, k)
    for _ in range(3):
        out = moe.moe_microscale_ffn(h, layer, ids, w, residual=r, workspace=work)
        assert torch.equal(out, want.to(torch.bfloat16))
    assert moe.moe_read_device_status(work) == 0
    if not res:
        at = torch.where(rr < 0, 0, rr).long()
        exact = (torch.where((rr < 0).unsqueeze(-1), 0.0, y[at].double()) * w.double().unsqueeze(-1)).sum(1)
        err = [float((v.double() - exact).norm() / exact.norm()) for v in (out, half)]
        assert err[0] <= 2.0 ** -9 and err[0] < err[1], err


@pytest.mark.parametrize("rows", [30, 60])
def test_gated_product_of_blocks_without_a_value(rows):
    """A NaN block (scale byte 255) in a row of x reaches all of that row's blocks, one in a gate or
    an up channel that channel's block in its expert's rows: scale byte 255 and codes 0 there,
    every other block as without them.  Both tiles."""
    g = gen(rows)
    E, I, K = 2, 96, 160
    sizes = [rows // 2, rows - rows // 2]
    offsets = torch.tensor([0, sizes[0], rows], dtype=torch.int32).cuda()
    code = lambda *shape: torch.randint(0, 16, shape, generator=g, dtype=torch.uint8)
    xcode, wcode = code(rows, K), code(E, 2 * I, K)
    xbyte = torch.full((rows, K // 32), 123, dtype=torch.uint8)
    wbyte = torch.full((E, 2 * I, K // 32), 126, dtype=torch.uint8)

    def run():
        args = [t.cuda() for t in ref.pack(xcode, xbyte) + ref.pack(wcode, wbyte)]
        work = torch.zeros(256, dtype=torch.uint8, device="cuda")
        c, s = moe.moe_microscale_gated_product(*args, offsets=offsets, workspace=work)
        assert moe.moe_read_device_status(work) == 0
        return c.cpu().reshape(rows, I // 32, 16), s.cpu()[:, :I // 32]
    want_c, want_s = run()
    assert int((want_s == 255).sum()) == 0
    xbyte[3, 4], xbyte[rows - 1, 0] = 255, 255
    wbyte[0, 40, 1], wbyte[1, I + 95, 3] = 255, 255  # expert 0's gate 40, expert 1's up 95
    bad = torch.zeros((rows, I // 32), dtype=torch.bool)
    bad[3], bad[rows - 1] = True, True
    bad[:sizes[0], 1], bad[sizes[0]:, 2] = True, True
    got_c, got_s = run()
    assert torch.equal(got_s == 255, bad) and int(got_c[bad].sum()) == 0
    assert torch.equal(got_s[~bad], want_s[~bad]) and torch.equal(got_c[~bad], want_c[~bad])


@pytest.mark.parametrize("rows", [32, 64])
def test_gated_product_of_infinities(rows):
    """g or u past fp32's range: the block is a NaN block; the row's others are not."""
    I, K = 64, 32
    xc, xs = ref.pack(torch.full((rows, K), 2, dtype=torch.uint8), torch.full((rows, 1), 127, dtype=torch.uint8))
    byte = torch.full((2 * I, 1), 127, dtype=torch.uint8)
    byte[3] = 252  # gate 3: 32 * 6 * 2^125 overflows; 2^125 itself does not
    byte[I + 40] = 252
    wc, ws = ref.pack(torch.full((2 * I, K), 7, dtype=torch.uint8), byte)
    for gate, up, want in ((True, False, [255, None]), (False, True, [None, 255])):
        s = ws.clone()
        if not gate:
            s[3] = ws[0]
        if not up:
            s[I + 40] = ws[0]
        c, sc = (t.cpu() for t in moe.moe_microscale_gated_product(xc.cuda(), xs.cuda(), wc.cuda(), s.cuda()))
        for b, w in enumerate(want):
            if w == 255:
                assert bool((sc[:, b] == 255).all()) and int(c[:, 16 * b:16 * b + 16].sum()) == 0
            else:
                v = ref.values(c[:, 16 * b:16 * b + 16].contiguous(), sc[:, b:b + 1])  # 192 * 192 = 36864 to 4 bits
                assert bool(((v - 36864).abs() <= 0.25 * 36864).all())


@pytest.mark.parametrize("rows", [32, 64])
def test_gated_product_far_below_zero(rows):
    """Row m has m ones: g = -4 m, u = 6 m 2^100.  SiLU(g) u is 4-bit rounded (a quarter of it at
    most), or 0 where the reciprocal is: below g = -87 and under 2^-119 |u|."""
    K, I = 32, 32
    m = torch.arange(rows) % 32 + 1
    code = torch.where(torch.arange(K) < m.unsqueeze(1), 2, 0).to(torch.uint8)  # 1.0
    xc, xs = ref.pack(code, torch.full((rows, 1), 127, dtype=torch.uint8))
    wcode = torch.cat((torch.full((I, K), 14), torch.full((I, K), 7))).to(torch.uint8)  # -4, 6
    byte = torch.cat((torch.full((I, 1), 127), torch.full((I, 1), 227))).to(torch.uint8)
    wc, ws = ref.pack(wcode, byte)
    c, s = moe.moe_microscale_gated_product(xc.cuda(), xs.cuda(), wc.cuda(), ws.cuda())
    got = ref.values(c.cpu(), s.cpu())
    g, u = -4.0 * m.double().unsqueeze(1), 6.0 * m.double().unsqueeze(1) * 2.0 ** 100
    p = (g * torch.exp(g) / (1 + torch.exp(g)) * u).expand(rows, I)
    flushed = (got == 0) & (g < -87) & (p.abs() <= 2.0 ** -119 * u)
    assert bool((((got - p).abs() <= (0.25 + 1e-4) * p.abs()) | flushed).all())
    assert bool((got[m <= 21] != 0).all())


def pitched(t, pad, shift):
    """The same matrix on the GPU with a longer pitch, NaN between the rows, and a base address off
    by `shift` elements."""
    R, C = t.shape
    buf = torch.full((R * (C + pad) + shift,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[shift:].view(R, C + pad)[:, :C]
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,k,E,H,pad,shift", [(1, 8, 128, 2048, 0, 0), (53, 5, 12, 608, 0, 0), (53, 5, 12, 608, 8, 8),
                                               (29, 18, 40, 544, 3, 1), (40, 32, 8, 96, 16, 0), (700, 3, 8, 1056, 1, 0)])
def test_quantise_into_sorted_rows_of_any_type_and_pitch(M, k, E, H, pad, shift, dtype):
    """Bit for bit the definition's codes at the rows of a token's routes, zeros in the rows of
    dropped ones; NaN and infinite blocks, blocks of zeros and of the largest values among them."""
    g = gen(M * H)
    ids = torch.randint(-1, E, (M, k), generator=g, dtype=torch.int32)
    x = torch.randn((M, H), generator=g) * torch.exp2(torch.randint(-8, 8, (M, 1), generator=g).float())
    x[0, :32], x[M // 2, -32:] = 0.0, torch.finfo(dtype).max
    x[M - 1, 40], x[M // 3, 5] = float("nan"), float("-inf")
    x = x.to(dtype)
    route_row = ref.plan(ids, E)[2]
    at, live = ref.at_rows(route_row)
    codes, scales = moe.moe_microscale_quantize(pitched(x, pad, shift), route_row=route_row.cuda())
    one_c, one_s = ref.pack(*ref.quantise(x))
    token = torch.arange(M).repeat_interleave(k)
    want_c = torch.zeros((M * k, H // 2), dtype=torch.uint8)
    want_s = torch.zeros((M * k, one_s.shape[1]), dtype=torch.uint8)
    want_c[at[live]], want_s[at[live]] = one_c[token[live]], one_s[token[live]]
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 32, 0, 1), (7, 480, 3, 0), (21, 2048, 1, 3), (130, 544, 8, 8), (5, 1568, 24, 0)])
def test_values_into_rows_of_any_pitch(rows, cols, pad, shift, dtype):
    """All scale bytes; nothing is written between the rows."""
    g = gen(rows * cols)
    code = torch.randint(0, 16, (rows, cols), generator=g, dtype=torch.uint8)
    byte = torch.randint(0, 256, (rows, cols // 32), generator=g, dtype=torch.uint8)
    c, s = ref.pack(code, byte)
    buf = torch.full((rows * (cols + pad) + shift + 5,), 77.0, dtype=dtype, device="cuda")
    out = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    moe.moe_microscale_dequantize(c.cuda(), s.cuda(), out=out)
    want = ref.values(c, s).to(dtype)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0, 1e30, -1e30), want.nan_to_num(0.0, 1e30, -1e30))
    out.fill_(77.0)
    assert bool((buf == 77.0).all())


@pytest.mark.parametrize("M,k,res", [(20, 9, True), (7, 17, True), (12, 18, False), (20, 18, True), (9, 32, True), (64, 32, False)])
def test_step_of_many_slots(M, k, res):
    """More than 8 slots, and past 18 the way back's other form, which does not begin early: the
    bits of the separate calls, in steps that follow one another."""
    E, H, I = 40, 288, 96
    layer = make_layer(E, H, I, seed=k)
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    work = moe.microscale_workspace(layer, M, k)
    hs, ids = [], []
    for _ in range(4):
        hs.append(torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16))
        ids.append(torch.randint(-1, E, (M, k), generator=g, device="cuda", dtype=torch.int32))
    w = torch.rand((M, k), generator=g, device="cuda")
    got = [moe.moe_microscale_ffn(h, layer, i, w, residual=h if res else None, workspace=work) for h, i in zip(hs, ids)]
    assert moe.moe_read_device_status(work) == 0
    for o, h, i in zip(got, hs, ids):
        assert torch.equal(o, parts(h, layer, i, w, residual=h if res else None))


@pytest.mark.parametrize("M,k", [(3, 4), (120, 8)])
def test_step_of_tokens_without_a_value(M, k):
    """A token with a NaN or an infinity: all of its own result is NaN, every other token's bits are
    as without it; a token whose routes are all dropped keeps its residual."""
    E, H, I = 16, 256, 96
    layer = make_layer(E, H, I, seed=9)
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((M, k), generator=g, device="cuda")
    h = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    res = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    ids[1] = -1
    work = moe.microscale_workspace(layer, M, k)
    want = moe.moe_microscale_ffn(h, layer, ids, w, residual=res, workspace=work)
    assert torch.equal(want[1], res[1])
    for value in (float("nan"), float("inf")):
        for token in (0, 1, M - 1):
            x = h.clone()
            x[token, 70] = value
            out = moe.moe_microscale_ffn(x, layer, ids, w, residual=res, workspace=work)
            keep = torch.arange(M, device="cuda") != token
            assert torch.equal(out[keep], want[keep])
            assert torch.equal(out[1], res[1])
            if token != 1:
                assert bool(torch.isnan(out[token]).all())
    assert moe.moe_read_device_status(work) == 0
