"""How the 16-bit grouped products' sums keep what the tensor core's accumulators would lose.

An accumulator truncates: what an MMA's 16 products add below the last of its 24 bits is gone, and
at worst each of the MMA's 17 addends is cut by 2^-23 of the largest.  So the sums of long
products and of long groups are split into chains, which are added up with rounding: of 256 of K (or
rows) for results in fp32 and for the 8-bit codes of f16 rows, of 8192 for 16-bit ones.
"""
import pytest
import torch

import grouped_ref as ref
from routed_expert_ffn_top_gb300 import moe

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
FINE, COARSE = 256, 8192
STEP = {BF16: 2.0 ** -8, F16: 2.0 ** -11}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def workspace():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def shares(n, value=1.0):
    """[n] with one nonzero in every 16 behind the first 16: what an MMA each adds."""
    v = torch.zeros(n, dtype=torch.float64, device="cuda")
    v[19::16] = value
    return v


def off(rows):
    return torch.tensor([0, rows], dtype=torch.int32, device="cuda")


def positive(shape, g, dtype, scale=1.0):
    return ((torch.rand(shape, generator=g, device="cuda") * 0.5 + 0.5) * scale).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("K,form", [(512, "plain"), (2048, "plain"), (5000, "plain"), (2048, "transposed"), (1000, "pair")])
def test_fp32_product_keeps_small_shares(K, form, rows, dtype):
    """2^24, and then a share of 1 in each MMA, half of its last bit: a chain of 16 MMAs loses at most
    15, and every addition of chains rounds by at most 1 (one accumulator would lose them all)."""
    n = 2 if form == "pair" else 1
    x = torch.cat([shares(K) for _ in range(n)])
    x[0] = 4096
    columns = torch.tensor([1.0, -1.0, 0.5, 2.0] * 4, dtype=torch.float64, device="cuda")
    w = [torch.ones((K, 16), dtype=torch.float64, device="cuda") * columns for _ in range(n)]
    w[0][0] *= 4096
    want = (x @ torch.cat(w)) / columns
    ws = [m.unsqueeze(0).to(dtype) for m in w]
    if form != "plain":
        ws = [m.transpose(1, 2).contiguous() for m in ws]
    work = workspace()
    got = moe.moe_grouped_product(x.to(dtype).expand(rows, -1).contiguous(), ws[0] if n == 1 else tuple(ws), off(rows), form != "plain",
                                  dtype=F32, workspace=work).double() / columns
    assert float(want[0]) == 2.0 ** 24 + n * len(range(19, K, 16))
    pieces = n * -(-K // FINE)
    assert float((got - want).abs().max()) <= 15 + (pieces - 1)
    assert moe.moe_read_device_status(work) == 0


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("code,top,tie", [(INT8, 127.0, 2.5), (E4M3, 448.0, 2.125)])
def test_codes_are_of_the_whole_sum(code, top, tie, rows):
    """g and u at a tie between two codes, and then shares of half their last bit: the first chain may
    lose its 15, those of the other seven put the sum past the tie."""
    H, I = 2048, 64
    x = shares(H, 2.0 ** -12)
    x[0] = 1
    w = torch.full((H, I), 2.0 ** -11, dtype=torch.float64, device="cuda")
    w[:, 0::32] = 0
    w[0] = tie
    w[0, 0::32] = top
    w[:, 1::2] *= -1
    want, scales = ref.quantise((x @ torch.cat((w, w.flip(1)), 1)).expand(rows, -1), code)
    rows_in = x.to(F16).expand(rows, -1).contiguous()
    work = workspace()
    got = moe.moe_grouped_gated_product(rows_in, w.unsqueeze(0).to(F16), w.flip(1).unsqueeze(0).to(F16).contiguous(), off(rows),
                                        checkpoint=code, workspace=work)
    assert torch.equal(got[2].cpu(), scales)
    assert torch.equal(got[1].cpu().view(torch.uint8), want.view(torch.uint8))
    assert moe.moe_read_device_status(work) == 0


@pytest.mark.parametrize("rows", [20, 300])
@pytest.mark.parametrize("K,form", [(16384, "plain"), (131072, "transposed"), (16384, "pair")])
def test_fp32_products_of_one_sign(K, form, rows):
    """Random values, all positive, so that every truncation pulls the same way: 16 MMAs of 17 addends a
    chain, each cut by at most 2^-23 of the sum, and the additions' 2^-24."""
    g = gen(K + rows)
    n = 2 if form == "pair" else 1
    x = positive((rows, n * K), g, F16)
    ws = [positive((1, 32, K), g, F16) for _ in range(n)]
    want = sum(x[:, i * K:(i + 1) * K].double() @ ws[i][0].double().t() for i in range(n))
    if form == "plain":
        ws = [w.transpose(1, 2).contiguous() for w in ws]
    got = moe.moe_grouped_product(x, ws[0] if n == 1 else tuple(ws), off(rows), form != "plain", dtype=F32, workspace=workspace())
    bound = 16 * 17 * 2.0 ** -23 + (n * K // FINE - 1) * 2.0 ** -24
    assert float(((got.double() - want) / want).abs().max()) <= bound


# a chain's 512 MMAs, and 127 additions of chains, in 2^20 of K
LONG = 512 * 17 * 2.0 ** -23 + 127 * 2.0 ** -24


@pytest.mark.parametrize("rows", [20, 80])
@pytest.mark.parametrize("transposed", [False, True])
def test_16_bit_products_of_the_longest_rows(transposed, rows):
    """K = 2^20, all positive: the chains' truncation and the result's rounding (one accumulator of 65,536
    MMAs is off by 7e-3)."""
    K = 1 << 20
    g = gen(rows)
    x, w = positive((rows, K), g, F16), positive((1, 32, K), g, F16, 2.0 ** -6)
    want = x.double() @ w[0].double().t()
    if not transposed:
        w = w.transpose(1, 2).contiguous()
    got = moe.moe_grouped_product(x, w, off(rows), transposed, workspace=workspace())
    assert float(((got.double() - want) / want).abs().max()) <= LONG + STEP[F16]


@pytest.mark.parametrize("rows", [20, 80])
def test_gated_products_of_the_longest_rows(rows):
    """H = 2^20.  p = SiLU(g) u: g's share counts 1 + g (1 - s) times, at most 1.28, u's once; the sigmoid
    within 2^-19 (1 + g), the rounding.  The way back: q times what the codes give."""
    H, I = 1 << 20, 32
    g = gen(rows + 1)
    x = positive((rows, H), g, F16, 2.0 ** -4)
    wg, wu = positive((1, H, I), g, F16, 2.0 ** -13), positive((1, H, I), g, F16, 2.0 ** -13)
    gx, ux = x.double() @ wg[0].double(), x.double() @ wu[0].double()
    work = workspace()
    p = moe.moe_grouped_gated_product(x, wg, wu, off(rows), workspace=work)
    want = ref.gate(gx, ux)
    assert float(((p.double() - want) / want).abs().max()) <= 2.28 * LONG + 2.0 ** -19 * (1 + float(gx.max())) + STEP[F16]
    with_codes, codes, scales = moe.moe_grouped_gated_product(x, wg, wu, off(rows), checkpoint=INT8, workspace=work)
    assert float(((with_codes.double() - want) / want).abs().max()) <= 2.28 * LONG + 2.0 ** -19 * (1 + float(gx.max())) + STEP[F16]
    wd = positive((1, I, H), g, F16, 2.0 ** -12)
    q = x.double() @ wd[0].double().t()
    ggu, _ = moe.moe_grouped_gated_product_grad(x, wd, off(rows), codes, scales, workspace=work)
    v = ref.values(codes.cpu(), scales.cpu()).cuda()
    want = ref.gate_grad(q, v[:, :I], v[:, I:])
    assert float(((ggu.double() - want) / want).abs().max()) <= LONG + 2.0 ** -18 * (1 + float(gx.max())) ** 2 + STEP[F16]
    assert moe.moe_read_device_status(work) == 0


@pytest.mark.parametrize("K,parts", [(16392, 1), (8200, 2), (5000, 2)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_bits_of_split_sums_do_not_depend_on_the_other_rows(out, K, parts):
    g = gen(K)
    rows = torch.randn((300, K * parts), generator=g, device="cuda").to(BF16)
    ws = [torch.randn((2, 72, K), generator=g, device="cuda").to(BF16) for _ in range(parts)]
    ws = ws[0] if parts == 1 else tuple(ws)
    y = moe.moe_grouped_product(rows, ws, torch.tensor([0, 200, 300], dtype=torch.int32, device="cuda"), True, dtype=out, workspace=workspace())
    for n in (1, 9):
        few = torch.cat((rows[50:50 + n], rows[220:221]))
        got = moe.moe_grouped_product(few, ws, torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda"), True, dtype=out,
                                      workspace=workspace())
        assert torch.equal(got[:n], y[50:50 + n]) and torch.equal(got[n], y[220])


@pytest.mark.parametrize("sizes,tail,N,K", [([1] * 8, 3, 200, 600), ([31, 0, 33, 64, 65], 1, 72, 776), ([255, 256, 257, 0, 513], 7, 264, 520),
                                            ([700, 5], 0, 40, 2048), ([97] * 40, 11, 520, 264)])
@pytest.mark.parametrize("form", ["plain", "transposed", "pair"])
def test_split_sums_of_ragged_groups(form, sizes, tail, N, K):
    """Small whole numbers, whose sums are exact in any order: several units a CTA pair, empty groups,
    dropped rows, widths that end inside tiles."""
    g = gen(N + K)
    n, parts = sum(sizes), 2 if form == "pair" else 1
    offsets = ref.groups(sizes)
    rows = torch.randint(-3, 4, (n + tail, K * parts), generator=g, device="cuda").to(BF16)
    rows[n:] = float("nan")
    E = len(sizes)
    ws = [torch.randint(-3, 4, (E, K, N) if form == "plain" else (E, N, K), generator=g, device="cuda").to(BF16) for _ in range(parts)]
    want = sum(ref.product(rows[:, i * K:(i + 1) * K].nan_to_num(0.0), w, offsets, form != "plain") for i, w in enumerate(ws))
    work = workspace()
    for _ in range(5):
        got = moe.moe_grouped_product(rows, ws[0] if parts == 1 else tuple(ws), offsets.cuda(), form != "plain", dtype=F32, workspace=work)
        assert torch.equal(got.double(), want)
    assert moe.moe_read_device_status(work) == 0


@pytest.mark.parametrize("sizes", [[2048], [300, 0, 5000, 17, 1100]])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_fp32_weight_grad_keeps_small_shares(dtype, sizes):
    """As of the products, along an expert's rows: the first row of each gives 2^24, then a row in 16 a share
    of 1."""
    offsets = ref.groups(sizes)
    x = torch.zeros((sum(sizes), 72), dtype=torch.float64, device="cuda")
    for _, lo, hi in ref.spans(offsets):
        if hi > lo:
            x[lo:hi] = shares(hi - lo).unsqueeze(1)
            x[lo] = 4096
    d = x[:, :40].contiguous()
    d[:, 1::2] *= -1
    work = workspace()
    got = moe.moe_grouped_weight_grad(x.to(dtype), d.to(dtype), offsets.cuda(), workspace=work).double()
    want = ref.weight_grad(x, d, offsets)
    for e, n in enumerate(sizes):
        assert float((got[e] - want[e]).abs().max()) <= (15 + (-(-n // FINE) - 1) if n else 0)
    assert moe.moe_read_device_status(work) == 0


@pytest.mark.parametrize("rows,E", [(127, 3), (128, 3), (129, 3), (129, 40), (1023, 150), (1024, 150)])
def test_tiles_at_the_borders_of_their_choice(rows, E):
    """All rows of one expert, and rows spread over all: around the numbers at which the tile changes."""
    g = gen(rows + E)
    x = torch.randint(-3, 4, (rows, 72), generator=g, device="cuda").to(BF16)
    w = torch.randint(-3, 4, (E, 72, 136), generator=g, device="cuda").to(BF16)
    work = workspace()
    for sizes in ([0] * (E - 1) + [rows], [rows // E + (e < rows % E) for e in range(E)]):
        offsets = ref.groups(sizes)
        got = moe.moe_grouped_product(x, w, offsets.cuda(), dtype=F32, workspace=work)
        assert torch.equal(got.double(), ref.product(x, w, offsets))
    assert moe.moe_read_device_status(work) == 0
