"""Refusals of the token sort and of the 4-bit entry points, without a GPU: what is wrong with the
arguments is reported before anything is launched."""
import ctypes

import pytest
import torch

import __graft_entry__ as entry
import tokens_ref as ref
from routed_expert_ffn_top_gb300 import moe

A = 1 << 20  # an aligned address; never dereferenced by validation
BAD, UNSUP, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return moe.lib()


def test_plan_refuses(lib):
    def plan(ids=A, M=4, k=2, E=8, off=A, rr=A, route=A):
        return lib.moe_token_plan(ids, M, k, E, off, rr, route, None)
    assert plan(M=-1) == BAD and plan(k=0) == BAD and plan(E=0) == BAD
    assert plan(k=33) == UNSUP and plan(E=1025) == UNSUP and plan(M=1 << 24, k=1) == UNSUP
    assert plan(ids=None) == BAD and plan(off=None) == BAD and plan(rr=None) == BAD and plan(route=None) == BAD
    assert plan(ids=A + 1) == BAD and plan(off=A + 2) == BAD


def test_sort_refuses(lib):
    def sort(x=A, ldx=64, dt=0, M=4, k=2, H=64, rr=A, rows=A, ldr=64):
        return lib.moe_token_sort(x, ldx, dt, M, k, H, rr, rows, ldr, None)
    assert sort(M=0, x=None, rows=None, rr=None) == moe.MOE_OK
    assert sort(dt=3) == BAD and sort(dt=-1) == BAD and sort(H=0) == BAD and sort(M=-1) == BAD and sort(k=0) == BAD
    assert sort(k=33) == UNSUP
    assert sort(x=None) == BAD and sort(rows=None) == BAD and sort(rr=None) == BAD
    assert sort(ldx=63) == BAD and sort(ldr=63) == BAD and sort(x=A + 1) == BAD and sort(dt=2, x=A + 2) == BAD


def test_unsort_and_gradients_refuse(lib):
    def unsort(rows=A, ldr=64, dt=0, M=4, k=2, H=64, rr=A, w=A, res=A, ldres=64, out=A, ldo=64):
        return lib.moe_token_unsort(rows, ldr, dt, M, k, H, rr, w, res, ldres, out, ldo, None)
    assert unsort(M=0, rows=None) == moe.MOE_OK
    assert unsort(rows=None) == BAD and unsort(out=None) == BAD and unsort(rr=None) == BAD
    assert unsort(ldres=10) == BAD and unsort(ldo=63) == BAD and unsort(w=A + 2) == BAD and unsort(dt=7) == BAD

    def grad(go=A, ldo=64, rows=A, ldr=64, dt=0, M=4, k=2, H=64, rr=A, w=A, g=A, ldg=64, gw=A):
        return lib.moe_token_unsort_grad(go, ldo, rows, ldr, dt, M, k, H, rr, w, g, ldg, gw, None)
    assert grad(M=0, go=None) == moe.MOE_OK
    assert grad(go=None) == BAD and grad(rows=None) == BAD and grad(g=None) == BAD and grad(gw=None) == BAD
    assert grad(gw=A + 1) == BAD and grad(ldg=1) == BAD
    assert lib.moe_token_sort_grad(None, 64, 0, 4, 2, 64, A, A, 64, None) == BAD


def test_quantise_refuses(lib):
    def quant(x=A, ldx=64, dt=0, rows=4, cols=64, rr=None, k=1, c=A, s=A):
        return lib.moe_microscale_quantize(x, ldx, dt, rows, cols, rr, k, c, s, None)
    assert quant(rows=0, x=None, c=None, s=None) == moe.MOE_OK
    assert quant(cols=33, ldx=64) == UNSUP and quant(cols=0) == BAD and quant(rows=-1) == BAD and quant(dt=5) == BAD
    assert quant(cols=(1 << 20) + 32, ldx=1 << 21) == UNSUP
    assert quant(x=None) == BAD and quant(c=None) == BAD and quant(s=None) == BAD
    assert quant(c=A + 8) == BAD and quant(s=A + 4) == BAD and quant(ldx=63) == BAD
    assert quant(rr=A, k=0) == BAD and quant(rr=A, k=33) == UNSUP and quant(rr=A + 2, k=2) == BAD
    assert lib.moe_microscale_dequantize(None, A, 4, 64, A, 64, 0, None) == BAD
    assert lib.moe_microscale_dequantize(A, A, 4, 48, A, 64, 0, None) == UNSUP
    assert lib.moe_microscale_dequantize(A, A, 4, 64, A, 32, 0, None) == BAD


def test_products_refuse(lib):
    def prod(xc=A, xs=A, rows=4, off=A, wc=A, ws=A, E=2, N=64, K=64, dt=0, y=A, ldy=64, work=A, n=256):
        return lib.moe_microscale_product(xc, xs, rows, off, wc, ws, E, N, K, dt, y, ldy, work, n, None)
    assert prod(rows=0, xc=None, wc=None, y=None) == moe.MOE_OK
    assert prod(rows=-1) == BAD and prod(E=0) == BAD and prod(N=0) == BAD and prod(K=0) == BAD and prod(dt=9) == BAD
    assert prod(K=40) == UNSUP and prod(E=1025) == UNSUP and prod(rows=1 << 24) == UNSUP and prod(E=1024, N=1 << 20) == UNSUP
    assert prod(off=None) == BAD and prod(work=None) == BAD and prod(n=255) == WS and prod(work=A + 8) == BAD
    for name in ("xc", "xs", "wc", "ws"):
        assert prod(**{name: None}) == BAD and prod(**{name: A + 8}) == BAD
    assert prod(y=None) == BAD and prod(ldy=63) == BAD

    def gated(N=64, c=A, s=A):
        return lib.moe_microscale_gated_product(A, A, 4, A, A, A, 2, N, 64, c, s, A, 256, None)
    assert gated(N=96) == UNSUP and gated(c=None) == BAD and gated(s=A + 1) == BAD


def test_expert_step_refuses(lib):
    w = moe.MicroscaleWeights(64, 32, 4, 0, A, A, A, A)
    need = lib.moe_microscale_workspace_bytes(ctypes.byref(w), 4, 2)
    assert need > 256 and need % 256 == 0
    assert lib.moe_microscale_workspace_bytes(ctypes.byref(w), -1, 2) == 0
    assert lib.moe_microscale_workspace_bytes(None, 4, 2) == 0

    def ffn(wt=w, h=A, M=4, k=2, ids=A, tw=A, out=A, work=A, n=need):
        return lib.moe_microscale_ffn(h, ctypes.byref(wt) if wt else None, M, k, ids, tw, None, out, work, n, None)
    assert ffn(M=0, h=None) == moe.MOE_OK
    assert ffn(wt=None) == BAD and ffn(h=None) == BAD and ffn(ids=None) == BAD and ffn(tw=None) == BAD and ffn(out=None) == BAD
    assert ffn(work=None) == BAD and ffn(work=A + 16) == BAD and ffn(n=need - 1) == WS and ffn(k=33) == UNSUP
    assert ffn(wt=moe.MicroscaleWeights(60, 32, 4, 0, A, A, A, A)) == UNSUP
    assert ffn(wt=moe.MicroscaleWeights(64, 16, 4, 0, A, A, A, A)) == UNSUP
    assert ffn(wt=moe.MicroscaleWeights(64, 32, 2000, 0, A, A, A, A)) == UNSUP


def test_pitch(lib):
    assert [moe.moe_microscale_pitch(c) for c in (32, 512, 544, 768, 2048)] == [16, 16, 32, 32, 64]
    assert moe.moe_microscale_pitch(33) == 0 and moe.moe_microscale_pitch(0) == 0


def test_binding_refuses(lib):
    x = torch.zeros((4, 64))
    rr = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        moe.moe_token_sort(x.double(), rr)
    with pytest.raises(TypeError):
        moe.moe_token_sort(x, rr.long())
    with pytest.raises(ValueError):
        moe.moe_token_sort(x, rr[:3])
    with pytest.raises(ValueError):
        moe.moe_token_sort(x, rr, stream=0)  # host memory
    with pytest.raises(ValueError):
        moe.moe_token_sort(x.t(), torch.zeros((64, 2), dtype=torch.int32))  # columns not contiguous
    with pytest.raises(ValueError):
        moe.moe_token_unsort(x[:1].expand(8, 64), rr)  # rows overlap
    with pytest.raises(ValueError):
        moe.moe_token_unsort(torch.zeros((8, 64)), rr, topk_weights=torch.zeros((4, 3)))
    with pytest.raises(TypeError):
        moe.moe_token_unsort(torch.zeros((8, 64)), rr, residual=x.to(torch.bfloat16))
    with pytest.raises(moe.MoeError):
        moe.moe_microscale_quantize(torch.zeros((4, 33)))
    with pytest.raises(ValueError):
        moe.moe_microscale_dequantize(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8))
    c, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 16), dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.moe_microscale_product(c, s, torch.zeros((8, 16), dtype=torch.uint8), torch.zeros((8, 16), dtype=torch.uint8))
    with pytest.raises(moe.MoeError):
        moe.moe_microscale_gated_product(c, s, torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 16), dtype=torch.uint8))


def test_reference_forms():
    """The tests' own plain forms, on values worked out by hand."""
    ids = torch.tensor([[2, 0], [9, 2], [0, -1]], dtype=torch.int32)
    offsets, row_route, route_row = ref.plan(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 4] and row_route.tolist() == [1, 4, 0, 3, -1, -1]
    assert route_row.tolist() == [[2, 0], [~4, 3], [1, ~5]]
    x = torch.zeros((1, 32))
    x[0, :8] = torch.tensor([4.0, 5.0, 2.5, -0.25, 0.75, 3.5, 0.2, 7.0])
    code, byte = ref.quantise(x)  # scale 2^0: ties 5 -> 4, 2.5 -> 2, 0.25 -> 0, 0.75 -> 1, 3.5 -> 4; 7 -> 6
    assert byte.tolist() == [[127]]
    assert ref.values(*ref.pack(code, byte))[0, :8].tolist() == [4.0, 4.0, 2.0, 0.0, 1.0, 4.0, 0.0, 6.0]
