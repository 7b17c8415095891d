"""Forms of the grouped calls that a program may use beside the usual ones, and what the training
example keeps and reports."""
import pytest
import torch

import grouped_ref as ref
from routed_expert_ffn_top_gb300 import moe
from test_gpu_grouped_use import BOUND, E4M3, F16, INT8, ex, gen, layer

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def workspace():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("sizes,tail,H,I", [([1], 0, 8, 32), ([16, 0, 1], 2, 72, 64), ([255, 256, 257, 0, 513], 7, 264, 160),
                                            ([97] * 40, 11, 520, 544), ([256] * 30, 0, 64, 1024), ([2, 0, 17, 9, 0, 0, 1, 30] * 8, 4, 1032, 480)])
def test_gate_gradient_without_p(sizes, tail, H, I, code):
    """The C entry's p may be NULL: the gradient of gate and up is bit for bit that with p, whose stores take
    their turns among the gradient's."""
    g = gen(H + I)
    n, E = sum(sizes) + tail, len(sizes)
    offsets = ref.groups(sizes).cuda()
    codes, scales = moe.moe_checkpoint_quantize(torch.randn((n, 2 * I), generator=g, device="cuda"), dtype=code)
    gy = torch.randn((n, H), generator=g, device="cuda").to(BF16)
    wd = torch.randn((E, I, H), generator=g, device="cuda").to(BF16)
    work = workspace()
    want, _ = moe.moe_grouped_gated_product_grad(gy, wd, offsets, codes, scales, workspace=work)
    for _ in range(3):
        got = torch.full_like(want, float("nan"))
        rc = moe.lib().moe_grouped_gated_product_grad(
            gy.data_ptr(), H, n, moe.MOE_DT_BF16, offsets.data_ptr(), wd.data_ptr(), E, I, H,
            moe.MOE_CODE_INT8 if code is INT8 else moe.MOE_CODE_E4M3, codes.data_ptr(), scales.data_ptr(), got.data_ptr(), None,
            work.data_ptr(), work.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == moe.MOE_OK
        assert torch.equal(got, want)
    assert not want[n - tail:].any()
    assert moe.moe_read_device_status(work) == 0


def test_16_bit_weight_grad_of_the_longest_groups():
    """2^20 rows of one sign into f16: 512 MMAs of 17 addends a chain, each cut by at most 2^-23 of the sum, 127
    additions, the rounding.  (One chain of 65,536 MMAs pulls all results down by 5e-3.)"""
    g = gen(3)
    R = 1 << 20
    x = (torch.rand((R, 40), generator=g, device="cuda") * 0.5 + 0.5).to(F16)
    d = ((torch.rand((R, 24), generator=g, device="cuda") * 0.5 + 0.5) * 2.0 ** -6).to(F16)
    want = x.double().t() @ d.double()
    got = moe.moe_grouped_weight_grad(x, d, dtype=F16, workspace=workspace())[0]
    assert float(((got.double() - want) / want).abs().max()) <= 512 * 17 * 2.0 ** -23 + 127 * 2.0 ** -24 + 2.0 ** -11


@pytest.mark.parametrize("M,H,I,E,k", [(64, 512, 256, 8, 2), (77, 160, 96, 6, 3)])
def test_memory_kept_is_as_stated(M, H, I, E, k):
    """The bytes that the function keeps for its way back, beside the weights and the plan."""
    x, w, wg, wu, wd, ids, d = layer(M, H, I, E, k, BF16, M)
    offsets, _, rr = moe.moe_token_plan(ids, E)
    leaves = [t.detach().requires_grad_() for t in (x, w, wg, wu, wd)]
    there = {t.data_ptr() for t in (*leaves, offsets, rr)}
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        out = ex.ExpertMLP.apply(*leaves, offsets, rr, INT8, workspace())
    new = {t.data_ptr(): t.numel() * t.element_size() for t in kept if t.data_ptr() not in there}
    assert sum(new.values()) == ex.memory(M, H, I, k)[1]
    out.backward(d)


@pytest.mark.parametrize("code", [E4M3, INT8])
def test_status_is_zero_after_a_training_pass(code):
    x, w, wg, wu, wd, ids, d = layer(300, 128, 96, 6, 2, BF16, 11, 0.1)
    offsets, _, rr = moe.moe_token_plan(ids, 6)
    leaves = [t.detach().requires_grad_() for t in (x, w, wg, wu, wd)]
    work = workspace()
    ex.ExpertMLP.apply(*leaves, offsets, rr, code, work).backward(d)
    assert moe.moe_read_device_status(work) == 0


def test_gradient_against_the_functions_own_differences():
    """Along the gradient of x, from two outputs of the kernels: each is off by at most BOUND of its norm; the
    gradient by the 8-bit checkpoints, 0.06 of its norm at most (as in the test with and without them); the
    curvature's share is about step^2.  The direction is what the two inputs, rounded to f16, are apart."""
    x, w, wg, wu, wd, ids, d = layer(400, 128, 96, 4, 2, F16, 6)
    offsets, _, rr = moe.moe_token_plan(ids, 4)
    work = workspace()
    leaf = x.detach().requires_grad_()
    ex.ExpertMLP.apply(leaf, w, wg, wu, wd, offsets, rr, INT8, work).backward(d)
    g = leaf.grad.double()
    step = 2.0 ** -3
    v = g / g.square().mean().sqrt()
    ends = [(x.double() + s * step * v).to(F16) for s in (1, -1)]
    outs = [ex.ExpertMLP.apply(e, w, wg, wu, wd, offsets, rr, INT8, work).double() for e in ends]
    apart = ends[0].double() - ends[1].double()
    got = float(((outs[0] - outs[1]) * d.double()).sum())
    want = float((g * apart).sum())
    noise = BOUND[F16] * float((outs[0].norm() + outs[1].norm()) * d.double().norm())
    assert noise <= 0.05 * want  # the two outputs are far enough apart to say something
    assert abs(got - want) <= 0.06 * float(g.norm() * apart.norm()) + noise + step ** 2 * want
