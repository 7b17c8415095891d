"""16-bit grouped products, their gradients and 8-bit checkpoints against plain fp64 forms.

Operands of small whole numbers: every partial sum is a whole number below 2^24, which fp32 holds
exactly in any order, so fp32 results must be equal and 16-bit ones their rounding.  Elsewhere
tolerances count roundings: half a step of the result's type, and for what is computed in fp32
from exact sums the bounds written at the tests.
"""
import pytest
import torch

import grouped_ref as ref
import tokens_ref
from routed_expert_ffn_top_gb300 import moe

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(shape, g, most, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dtype)


def status(work):
    return moe.moe_read_device_status(work)


def workspace():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


# group sizes around both tiles' rows and the steps of a group's division, empty groups, one row
# each, more tiles than SMs; the last number is rows past the last group.  Widths inside, at and
# past the channel tiles; lengths below a K step, inside a stage, across stages.
SHAPES = [([1], 0, 8, 8), ([3, 0, 1], 2, 64, 72), ([0, 0, 5], 0, 136, 128), ([1] * 8, 3, 200, 264), ([31, 32, 33, 64, 65], 1, 72, 136),
          ([127, 128, 129], 5, 256, 192), ([255, 256, 257, 0, 513], 7, 264, 200), ([300], 0, 512, 520), ([40] * 30, 9, 96, 160),
          ([700, 5], 0, 40, 768), ([20000], 0, 16, 32), ([97] * 40, 11, 520, 136), ([2, 0, 17, 9, 0, 0, 1, 30] * 8, 4, 1000, 1032)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("form", ["plain", "transposed", "pair", "pair plain"])
@pytest.mark.parametrize("sizes,tail,N,K", SHAPES)
def test_product_exact_sums(sizes, tail, N, K, form, dtype):
    g = gen(N * K + len(sizes))
    E, parts, transposed = len(sizes), 2 if form.startswith("pair") else 1, form in ("transposed", "pair")
    offsets = ref.groups(sizes)
    n = sum(sizes)
    rows = ints((n + tail, K * parts), g, 3, dtype)
    rows[n:] = float("nan")  # dropped routes' rows: never read into a result
    ws = [ints((E, N, K) if transposed else (E, K, N), g, 3, dtype) for _ in range(parts)]
    want = sum(ref.product(rows[:, i * K:(i + 1) * K].nan_to_num(0.0), w, offsets, transposed) for i, w in enumerate(ws))
    work = workspace()
    weights = ws[0] if parts == 1 else tuple(ws)
    for out in (F32, BF16, F16):
        y = torch.full((n + tail, N + 24), float("nan"), dtype=out, device="cuda")
        moe.moe_grouped_product(rows, weights, offsets.cuda(), transposed, out=y[:, 8:8 + N], workspace=work)
        assert torch.equal(y[:, 8:8 + N], want.to(F32).to(out))
        assert torch.isnan(y[:, :8].float()).all() and torch.isnan(y[:, 8 + N:].float()).all()
    y = moe.moe_grouped_product(rows, weights, offsets.cuda(), transposed)
    assert y.dtype is dtype and torch.equal(y, want.to(F32).to(dtype))
    assert status(work) == 0


@pytest.mark.parametrize("rows,out", [(80, BF16), (48, F16), (112, F32), (208, BF16)])
def test_product_of_many_short_units(rows, out):
    """Few MMAs a unit, odd numbers of 16-row steps: every store's staging memory is still in use when
    the next unit's results come."""
    g = gen(rows)
    offsets = ref.groups([rows] * 48)
    x, w = ints((48 * rows, 32), g, 3, BF16), ints((48, 32, 2048), g, 3, BF16)
    want = ref.product(x, w, offsets).to(F32).to(out)
    work, y = workspace(), torch.empty((48 * rows, 2048), dtype=out, device="cuda")
    for _ in range(20):
        y.fill_(float("nan"))
        moe.moe_grouped_product(x, w, offsets.cuda(), out=y, workspace=work)
        assert torch.equal(y, want)


def test_product_any_result_pitch():
    """Rows of y that allow no wide stores: odd pitch and offset."""
    g = gen(3)
    offsets = ref.groups([50, 300])
    rows, w = ints((350, 64), g, 3, BF16), ints((2, 64, 200), g, 3, BF16)
    want = ref.product(rows, w, offsets)
    for dtype in (BF16, F32):
        y = torch.full((360, 211), 7.0, dtype=dtype, device="cuda")
        moe.moe_grouped_product(rows, w, offsets.cuda(), out=y[3:353, 5:205], workspace=workspace())
        assert torch.equal(y[3:353, 5:205], want.to(dtype))
        y[3:353, 5:205] = 7.0
        assert (y == 7.0).all()


def test_product_operand_pitch():
    g = gen(4)
    offsets = ref.groups([50, 0, 300])
    wide, w = ints((350, 256), g, 3, BF16), ints((3, 64, 96), g, 3, BF16)
    rows = wide[:, 40:104]
    got = moe.moe_grouped_product(rows, w, offsets.cuda(), dtype=F32, workspace=workspace())
    assert torch.equal(got.double(), ref.product(rows, w, offsets))


def test_product_one_group():
    g = gen(5)
    rows, w = ints((77, 72), g, 3, F16), ints((72, 40), g, 3, F16)
    want = rows.double() @ w.double()
    assert torch.equal(moe.moe_grouped_product(rows, w, dtype=F32).double(), want)
    assert torch.equal(moe.moe_grouped_product(rows, w.unsqueeze(0), dtype=F32).double(), want)
    got = moe.moe_grouped_weight_grad(rows, ints((77, 40), gen(6), 3, F16))
    assert torch.equal(got[0].double(), rows.double().t() @ ints((77, 40), gen(6), 3, F16).double())


def test_product_many_experts():
    g = gen(7)
    sizes = torch.randint(0, 5, (1024,), generator=torch.Generator().manual_seed(1)).tolist()
    offsets = ref.groups(sizes)
    rows, w = ints((sum(sizes) + 6, 40), g, 3, BF16), ints((1024, 40, 24), g, 3, BF16)
    got = moe.moe_grouped_product(rows, w, offsets.cuda(), dtype=F32, workspace=workspace())
    assert torch.equal(got.double(), ref.product(rows, w, offsets))
    d = ints((len(rows), 24), g, 3, BF16)
    got = moe.moe_grouped_weight_grad(rows, d, offsets.cuda(), workspace=workspace())
    assert torch.equal(got.double(), ref.weight_grad(rows, d, offsets))


def test_product_bits_do_not_depend_on_the_other_rows():
    """A row alone (small tile), among few, and among many (large tile) gives the same bits."""
    g = gen(8)
    rows = torch.randn((900, 1000), generator=g, device="cuda").to(BF16)
    w = torch.randn((2, 1000, 264), generator=g, device="cuda").to(BF16)
    d = torch.randn((2, 264, 1000), generator=g, device="cuda").to(BF16)
    for weights, t in ((w, False), (d, True)):
        y = moe.moe_grouped_product(rows, weights, ref.groups([400, 500]).cuda(), t, dtype=F32)
        for n in (1, 3, 30, 200):
            off = torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda")
            part = torch.cat((rows[100:100 + n], rows[700:701]))
            got = moe.moe_grouped_product(part, weights, off, t, dtype=F32)
            assert torch.equal(got[:n], y[100:100 + n]) and torch.equal(got[n], y[700])


# ---------------------------------------------------------------------------------- weights
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("sizes,tail,N,K", SHAPES)
def test_weight_grad_exact_sums(sizes, tail, N, K, dtype, out):
    g = gen(N + K + len(sizes))
    offsets = ref.groups(sizes)
    n = sum(sizes)
    rows, grads = ints((n + tail, K), g, 2, dtype), ints((n + tail, N), g, 2, dtype)
    rows[n:], grads[n:] = float("nan"), float("inf")
    want = ref.weight_grad(rows, grads, offsets).to(F32).to(out)
    got = torch.full((len(sizes), K, N), float("nan"), dtype=out, device="cuda")
    work = workspace()
    moe.moe_grouped_weight_grad(rows, grads, offsets.cuda(), out=got, workspace=work)
    assert torch.equal(got, want)
    assert status(work) == 0


def test_weight_grad_keeps_a_bad_row_within_its_group():
    """Rows of NaN and infinities in one expert's group: the neighbours' steps that read them too
    are not touched."""
    g = gen(9)
    sizes = [17, 5, 130, 1, 0, 40]
    offsets = ref.groups(sizes)
    rows, grads = ints((sum(sizes), 72), g, 3, BF16), ints((sum(sizes), 136), g, 3, BF16)
    want = ref.weight_grad(rows, grads, offsets)
    rows[17:22], grads[17:22] = float("nan"), float("inf")
    rows[152], grads[152] = float("inf"), float("nan")
    got = moe.moe_grouped_weight_grad(rows, grads, offsets.cuda(), workspace=workspace())
    for e in (0, 2, 4, 5):
        assert torch.equal(got[e].double(), want[e])
    assert torch.isnan(got[1]).all() and torch.isnan(got[3]).all()


def test_weight_grad_of_long_groups():
    """65,536 rows in one group.  fp32: chains of 32 MMAs, each of whose additions truncates by at most
    2^-23 of the sum so far, added up by 127 rounded additions of at most 2^-24: 32 2^-23 + 127 2^-24 of
    the 2-norm (one chain of 4096 MMAs would be off by up to 4096 2^-23).  16 bits: chains of 512 MMAs,
    seven additions, and the result's rounding, 2^-8."""
    g = gen(13)
    rows = torch.randn((65536 + 77, 72), generator=g, device="cuda").to(BF16)
    grads = torch.randn((65536 + 77, 40), generator=g, device="cuda").to(BF16)
    offsets = torch.tensor([0, 30, 65566, 65613], dtype=torch.int32)
    got = moe.moe_grouped_weight_grad(rows, grads, offsets.cuda(), workspace=workspace())
    want = ref.weight_grad(rows, grads, offsets)
    for e in range(3):
        assert float((got[e].double() - want[e]).norm()) <= (32 * 2.0 ** -23 + 127 * 2.0 ** -24) * float(want[e].norm())
    got = moe.moe_grouped_weight_grad(rows, grads, offsets.cuda(), dtype=BF16, workspace=workspace())
    for e in range(3):
        bound = 512 * 2.0 ** -23 + 7 * 2.0 ** -24 + 2.0 ** -8
        assert float((got[e].double() - want[e]).norm()) <= bound * float(want[e].norm())


@pytest.mark.parametrize("rows", (20, 900))
def test_some_of_a_layers_experts(rows):
    """Offsets of experts in the middle of the rows: the rows of others are zero, and add to nothing."""
    g = gen(14)
    lo, mid, hi = rows // 4, rows // 2, rows - 3
    offsets = torch.tensor([lo, mid, mid, hi], dtype=torch.int32)
    x, w, v = ints((rows, 64), g, 3, BF16), ints((3, 64, 32), g, 3, BF16), ints((3, 64, 32), g, 3, BF16)
    full = torch.tensor([0, lo, mid, mid, hi], dtype=torch.int32)
    nothing = torch.zeros((1, 64, 32), dtype=BF16, device="cuda")
    whole_w, whole_v = torch.cat((nothing, w)), torch.cat((nothing, v))
    work = workspace()
    assert torch.equal(moe.moe_grouped_product(x, w, offsets.cuda(), workspace=work),
                       moe.moe_grouped_product(x, whole_w, full.cuda(), workspace=work))
    got = moe.moe_grouped_gated_product(x, w, v, offsets.cuda(), checkpoint=torch.int8, workspace=work)
    want = moe.moe_grouped_gated_product(x, whole_w, whole_v, full.cuda(), checkpoint=torch.int8, workspace=work)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    down, whole_down = w.transpose(1, 2).contiguous(), whole_w.transpose(1, 2).contiguous()
    got = moe.moe_grouped_gated_product_grad(x, down, offsets.cuda(), *got[1:], workspace=work)
    want = moe.moe_grouped_gated_product_grad(x, whole_down, full.cuda(), *want[1:], workspace=work)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(moe.moe_grouped_weight_grad(x, x, offsets.cuda(), workspace=work),
                       moe.moe_grouped_weight_grad(x, x, full.cuda(), workspace=work)[1:])


def test_weight_grad_of_column_halves():
    """The two halves of one matrix of gradients, by their pitch."""
    g = gen(10)
    offsets = ref.groups([100, 28])
    rows, both = ints((128, 64), g, 3, F16), ints((128, 176), g, 3, F16)
    for part in (both[:, :88], both[:, 88:]):
        got = moe.moe_grouped_weight_grad(rows, part, offsets.cuda(), workspace=workspace())
        assert torch.equal(got.double(), ref.weight_grad(rows, part, offsets))


def test_no_rows():
    w = torch.ones((3, 16, 32), dtype=BF16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    rows = torch.empty((0, 16), dtype=BF16, device="cuda")
    assert moe.moe_grouped_product(rows, w, off).shape == (0, 32)
    p, codes, scales = moe.moe_grouped_gated_product(rows, w, w, off, checkpoint=INT8)
    assert p.shape == (0, 32) and codes.shape == (0, 64)
    d = torch.empty((0, 24), dtype=BF16, device="cuda")
    got = moe.moe_grouped_weight_grad(rows, d, off, out=torch.ones((3, 16, 24), device="cuda"))
    assert (got == 0).all()
    # rows, but all of dropped routes
    rows = torch.full((5, 16), float("nan"), dtype=BF16, device="cuda")
    assert (moe.moe_grouped_product(rows, w, off) == 0).all()
    assert (moe.moe_grouped_weight_grad(rows, rows, off) == 0).all()


# ------------------------------------------------------------------------------------ gated
GATED = [([1], 0, 8, 32), ([3, 0, 1], 2, 72, 64), ([31, 32, 33, 64, 65], 1, 136, 96), ([255, 256, 257, 0, 513], 7, 264, 160),
         ([97] * 40, 11, 520, 352), ([2, 0, 17, 9, 0, 0, 1, 30] * 8, 4, 1032, 480)]


def gated_inputs(sizes, tail, H, I, dtype, seed=0):
    """Rows and weights with exact sums, |g| up to about 10."""
    g = gen(H * I + seed)
    n = sum(sizes)
    rows = ints((n + tail, H), g, 2, dtype)
    rows[n:] = float("nan")
    scale = 2.0 ** -4
    return (rows, ints((len(sizes), H, I), g, 2, dtype) * scale, ints((len(sizes), H, I), g, 2, dtype) * scale,
            ref.groups(sizes))


def close(got, want, bound):
    """Within `bound`, elementwise."""
    bad = (got.double() - want).abs() > bound
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype,code", [(BF16, None), (BF16, E4M3), (BF16, INT8), (F16, E4M3), (F16, INT8)])
@pytest.mark.parametrize("sizes,tail,H,I", GATED)
def test_gated_product_and_checkpoint(sizes, tail, H, I, dtype, code):
    rows, wg, wu, offsets = gated_inputs(sizes, tail, H, I, dtype)
    n = sum(sizes)
    clean = rows.nan_to_num(0.0)
    gx, ux = ref.product(clean, wg, offsets), ref.product(clean, wu, offsets)
    work = workspace()
    out = torch.full((n + tail, I + 16), float("nan"), dtype=dtype, device="cuda")
    got = moe.moe_grouped_gated_product(rows, wg, wu, offsets.cuda(), checkpoint=code, out=out[:, :I], workspace=work)
    assert status(work) == 0
    p = got if code is None else got[0]
    want = ref.gate(gx, ux)
    # the sigmoid within 2^-20 (1 + |g| / 4), two products, the rounding; 2^-25 half the smallest f16
    close(p, want, want.abs() * (HALF[dtype] + 2.0 ** -19 * (1 + gx.abs())) + 2.0 ** -25)
    assert torch.isnan(out[:, I:].float()).all()
    assert (p[n:] == 0).all()
    if code is not None:
        # g and u are exact in fp32, so every code is decided
        codes, scales = ref.quantise(torch.cat((gx, ux), 1), code)
        codes[n:], scales[n:] = torch.zeros((), dtype=code), 0
        assert torch.equal(got[2].cpu(), scales)
        assert torch.equal(got[1].cpu().view(torch.uint8), codes.view(torch.uint8))


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("sizes,tail,H,I", GATED)
def test_gated_product_grad(sizes, tail, H, I, dtype, code):
    g = gen(H + I)
    n, E = sum(sizes), len(sizes)
    offsets = ref.groups(sizes)
    gu = torch.randn((n + tail, 2 * I), generator=g, device="cuda") * 2
    codes, scales = moe.moe_checkpoint_quantize(gu, dtype=code)
    v = ref.values(codes.cpu(), scales.cpu()).cuda()
    gy, wd = ints((n + tail, H), g, 2, dtype), ints((E, I, H), g, 2, dtype) * 2.0 ** -4
    gy[n:] = float("nan")
    work = workspace()
    ggu, p = moe.moe_grouped_gated_product_grad(gy, wd, offsets.cuda(), codes, scales, workspace=work)
    assert status(work) == 0
    assert (ggu[n:] == 0).all() and (p[n:] == 0).all()
    q = ref.product(gy.nan_to_num(0.0), wd, offsets, True)[:n]
    gx, ux = v[:n, :I], v[:n, I:]
    want = ref.gate_grad(q, gx, ux)
    # s (1 + g (1 - s)) as s + g s (1 - s): each factor within 2^-20 (1 + |g|) of itself, the sum's terms
    # add up to at most (1 + |g|) s; then the rounding
    slack = 2.0 ** -18 * (1 + gx.abs()) ** 2
    bound = torch.cat(((q * ux).abs() * slack, q.abs() * gx.abs() * slack), 1) + want.abs() * HALF[dtype] + 2.0 ** -25
    close(ggu[:n], want, bound)
    want = ref.gate(gx, ux)
    close(p[:n], want, want.abs() * (HALF[dtype] + 2.0 ** -19 * (1 + gx.abs())) + 2.0 ** -25)


def test_gated_any_result_pitch():
    """Rows of p that allow no wide stores."""
    rows, wg, wu, offsets = gated_inputs([40, 0, 300], 3, 136, 96, BF16)
    want = moe.moe_grouped_gated_product(rows, wg, wu, offsets.cuda(), workspace=workspace())
    p = torch.full((350, 107), 7.0, dtype=BF16, device="cuda")
    moe.moe_grouped_gated_product(rows, wg, wu, offsets.cuda(), out=p[2:345, 5:101], workspace=workspace())
    assert torch.equal(p[2:345, 5:101], want)
    p[2:345, 5:101] = 7.0
    assert (p == 7.0).all()


def test_gated_grad_with_given_results():
    """Results of the caller's own, p and the gradient side by side in one buffer."""
    g = gen(12)
    offsets = ref.groups([30, 200])
    gy, wd = ints((230, 64), g, 3, BF16), ints((2, 96, 64), g, 3, BF16)
    codes, scales = moe.moe_checkpoint_quantize(torch.randn((230, 192), generator=g, device="cuda"), dtype=INT8)
    want = moe.moe_grouped_gated_product_grad(gy, wd, offsets.cuda(), codes, scales, workspace=workspace())
    buf = torch.full((231, 288), 7.0, dtype=BF16, device="cuda").reshape(-1)
    ggu, p = buf[8:8 + 230 * 192].reshape(230, 192), buf[16 + 230 * 192:16 + 230 * 288].reshape(230, 96)
    moe.moe_grouped_gated_product_grad(gy, wd, offsets.cuda(), codes, scales, grad_gate_up=ggu, p=p, workspace=workspace())
    assert torch.equal(ggu, want[0]) and torch.equal(p, want[1])
    assert (buf[:8] == 7.0).all() and (buf[16 + 230 * 288:] == 7.0).all()


def test_gated_far_values():
    """Gates far from zero, infinite and NaN ones: as the formula's limits, no NaN of its own."""
    rows = torch.eye(8, dtype=BF16, device="cuda")
    g = torch.tensor([0.0, 50.0, -50.0, 120.0, -120.0, 3e38, float("inf"), float("nan")], device="cuda")
    wg = torch.zeros((1, 8, 32), dtype=BF16, device="cuda")
    wg[0] = g.unsqueeze(1)
    wu = torch.full((1, 8, 32), 2.0, dtype=BF16, device="cuda")
    # one row a gate, so that no sum mixes them (0 times an infinity is a NaN)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(8):
        only = wg.clone()
        only[0, torch.arange(8) != i] = 0
        p, codes, scales = moe.moe_grouped_gated_product(rows[i:i + 1], only, wu, off, checkpoint=E4M3)
        x = only[0, i, 0].double()
        want = (x * torch.sigmoid(x) * 2.0).to(BF16)
        if i == 4:
            assert p.abs().max() < 1e-30
        elif torch.isnan(want):
            assert torch.isnan(p).all()
        else:
            close(p, want.double().expand(1, 32), want.double().abs() * 2.0 ** -7)
        bad = not torch.isfinite(only[0, i, 0])
        assert (int(scales[0, 0]) == 255) == bad and int(scales[0, 1]) != 255


# ------------------------------------------------------------------------------- checkpoints
def edge_rows(cols, dtype):
    """Blocks of zeros, ties, the largest codes' borders, subnormals, the largest values,
    infinities and NaN."""
    fi = torch.finfo(dtype)
    blocks = [torch.zeros(32), -torch.zeros(32), torch.arange(32) + 0.5, torch.linspace(-448, 448, 32),
              torch.cat((torch.tensor([448.0]), torch.arange(31) * 2.0 ** -10)), torch.cat((torch.tensor([449.0]), torch.arange(31.0))),
              torch.cat((torch.tensor([127.0]), torch.arange(31) + 0.5)), torch.cat((torch.tensor([127.5]), torch.arange(31) + 0.5)),
              torch.full((32,), fi.max), torch.full((32,), fi.smallest_normal), torch.full((32,), fi.smallest_normal / 8),
              torch.linspace(-1, 1, 32) * fi.smallest_normal, torch.cat((torch.tensor([float("inf")]), torch.ones(31))),
              torch.cat((torch.ones(31), torch.tensor([float("nan")]))), torch.cat((torch.tensor([-float("inf")]), -torch.ones(31)))]
    n = cols // 32
    return torch.stack([torch.cat([blocks[(i + s) % len(blocks)] for i in range(n)]) for s in range(len(blocks))]).to(dtype)


def same(a, b):
    """Equal, NaN for NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(0.0, 1e30, -1e30), b.nan_to_num(0.0, 1e30, -1e30))


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 64, 0), (7, 480, 0), (21, 2048, 0), (5, 544, 3), (2, 1568, 8), (130, 768, 0)])
def test_checkpoint_bit_for_bit(rows, cols, pad, dtype, code):
    g = torch.Generator().manual_seed(rows * cols)
    x = torch.cat((torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-8, 8, (rows, 1), generator=g).float()),
                   edge_rows(cols, dtype).float())).to(dtype)
    R = x.shape[0]
    buf = torch.full((R, cols + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = x.cuda()
    codes, scales = moe.moe_checkpoint_quantize(buf[:, :cols], dtype=code)
    wc, ws = ref.quantise(x, code)
    assert torch.equal(scales.cpu(), ws)
    assert torch.equal(codes.cpu().view(torch.uint8), wc.view(torch.uint8))
    want = ref.values(wc, ws)
    for out in (BF16, F16, F32):
        assert same(moe.moe_checkpoint_dequantize(codes, scales, dtype=out).cpu(), want.to(F32).to(out))
        y = torch.full((R, cols + pad), 7.0, dtype=out, device="cuda")
        moe.moe_checkpoint_dequantize(codes, scales, out=y[:, :cols])
        assert same(y[:, :cols].cpu(), want.to(F32).to(out)) and (y[:, cols:] == 7.0).all()


@pytest.mark.parametrize("code", [E4M3, INT8])
def test_checkpoint_every_bf16_value(code):
    """All 65536 bf16 patterns, each the largest of its block."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16).reshape(-1, 1)
    x = torch.cat((x, x.float().mul(0.4).to(BF16), torch.zeros((65536, 30), dtype=BF16)), 1)
    codes, scales = moe.moe_checkpoint_quantize(x.cuda(), dtype=code)
    wc, ws = ref.quantise(x, code)
    assert torch.equal(scales.cpu(), ws)
    assert torch.equal(codes.cpu().view(torch.uint8), wc.view(torch.uint8))


@pytest.mark.parametrize("code", [E4M3, INT8])
def test_checkpoint_error_is_half_a_step(code):
    """The bound that the format states, at random values over many powers of two."""
    g = gen(11)
    x = torch.randn((512, 1024), generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (512, 1024), generator=g, device="cuda").float())
    codes, scales = moe.moe_checkpoint_quantize(x, dtype=code)
    v = moe.moe_checkpoint_dequantize(codes, scales, dtype=F32).double()
    top = x.double().abs().reshape(512, -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(512, 1024)
    err = (v - x.double()).abs()
    if code is INT8:
        assert (err <= top / 127).all()
    else:
        # half a step of the code: 2^-4 of the value, or half the subnormal step 2^-9 2^X, 2^X < 2 top / 448
        assert (err <= torch.maximum(x.double().abs() * 2.0 ** -4, top * 2 / 448 * 2.0 ** -10)).all()


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("M,k,cols,dtype,pad", [(1, 1, 32, BF16, 0), (53, 5, 608, BF16, 0), (7, 32, 64, F16, 3), (300, 3, 1056, F32, 0)])
def test_checkpoint_into_sorted_rows(M, k, cols, dtype, pad, code):
    E = 12
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-1, E, (M, k), generator=g, dtype=torch.int32)
    x = torch.randn((M, cols), generator=g).to(dtype).cuda()
    rr = moe.moe_token_plan(ids.cuda(), E)[2]
    codes, scales = moe.moe_checkpoint_quantize(x, dtype=code)
    want = moe.moe_token_sort(moe.moe_checkpoint_dequantize(codes, scales, dtype=dtype), rr)
    assert torch.equal(moe.moe_checkpoint_dequantize(codes, scales, dtype=dtype, route_row=rr), want)
    out = torch.full((M * k, cols + pad), 7.0, dtype=dtype, device="cuda")
    moe.moe_checkpoint_dequantize(codes, scales, route_row=rr, out=out[:, :cols])
    assert torch.equal(out[:, :cols], want) and (out[:, cols:] == 7.0).all()
