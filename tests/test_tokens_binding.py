"""What the token and 4-bit calls check before anything is launched, on the CPU: a fake library
records the calls that would have reached the GPU."""
import ctypes

import pytest
import torch

import __graft_entry__ as entry
from routed_expert_ffn_top_gb300 import moe

A = 1 << 20  # an aligned address; never dereferenced by validation


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return moe.lib()


@pytest.mark.parametrize("name", ["gate_up_codes", "gate_up_scales", "down_codes", "down_scales"])
def test_expert_step_refuses_weights_before_a_launch(lib, name):
    """Launching here, without a device, would come back as MOE_ERR_CUDA."""
    for bad in (None, A + 8):
        w = moe.MicroscaleWeights(64, 32, 4, 0, A, A, A, A)
        setattr(w, name, bad)
        for M in (4, 200):  # both forms of the plan
            assert lib.moe_microscale_ffn(A, ctypes.byref(w), M, 2, A, A, None, A, A, 1 << 30, None) == moe.MOE_ERR_INVALID_ARG


class Recorder:
    """Stands in for the library: every call is recorded and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_bytes") else moe.MOE_OK
        return call


@pytest.fixture
def fake(monkeypatch):
    """The binding with host tensors in the place of the GPU's and the library recorded."""
    r = Recorder()
    monkeypatch.setattr(moe, "lib", lambda: r)
    monkeypatch.setattr(moe, "_raw_stream", lambda stream, device: 0)
    return r


def four_bit_layer(E=4, H=64, I=32, device="cpu"):
    layer = {"H": H, "I": I, "E": E}
    for name, n, cols in (("gate_up", 2 * I, H), ("down", H, I)):
        layer[name + "_codes"] = torch.zeros((E, n, cols // 2), dtype=torch.uint8, device=device)
        layer[name + "_scales"] = torch.zeros((E, n, 16), dtype=torch.uint8, device=device)
    return layer


def step_args(M=3, k=2, H=64, device="cpu"):
    return (torch.zeros((M, H), dtype=torch.bfloat16, device=device),
            torch.zeros((M, k), dtype=torch.int32, device=device), torch.zeros((M, k), device=device))


def launches(fake):
    return [n for n, _ in fake.calls if not n.endswith("_bytes")]


def test_step_takes_a_layer_of_its_own_device_only(fake):
    h, ids, w = step_args()
    work = torch.zeros(8192, dtype=torch.uint8)
    moe.moe_microscale_ffn(h, four_bit_layer(), ids, w, workspace=work)
    assert launches(fake) == ["moe_microscale_ffn"]
    fake.calls.clear()
    with pytest.raises(ValueError, match="meta"):
        moe.moe_microscale_ffn(h, four_bit_layer(device="meta"), ids, w, workspace=work)
    for name in ("gate_up_codes", "gate_up_scales", "down_codes", "down_scales"):
        layer = four_bit_layer()
        layer[name] = layer[name].to("meta")
        with pytest.raises(ValueError, match="meta"):
            moe.moe_microscale_ffn(h, layer, ids, w, workspace=work)
    assert launches(fake) == []


def quantised(*shape):
    return torch.zeros(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8), torch.zeros(shape[:-1] + (16,), dtype=torch.uint8)


BAD_WORKSPACES = [(torch.zeros(8192, dtype=torch.uint8, device="meta"), ValueError),
                  (torch.zeros(8192, dtype=torch.int32), TypeError),
                  (torch.zeros(16384, dtype=torch.uint8)[::2], ValueError)]


@pytest.mark.parametrize("work,error", BAD_WORKSPACES)
def test_a_workspace_is_contiguous_bytes_of_the_device(fake, work, error):
    h, ids, w = step_args()
    x, wt = quantised(3, 64), quantised(2, 64, 64)
    offsets = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(error):
        moe.moe_microscale_ffn(h, four_bit_layer(), ids, w, workspace=work)
    with pytest.raises(error):
        moe.moe_microscale_product(*x, *wt, offsets=offsets, workspace=work)
    with pytest.raises(error):
        moe.moe_microscale_gated_product(*x, *wt, offsets=offsets, workspace=work)
    assert launches(fake) == []


def test_rows_are_matrices(fake):
    """Codes [E,n,cols/2] of a layer are not rows: E of its E * n rows would come back."""
    layer, (c, s), wt = four_bit_layer(), quantised(3, 64), quantised(2, 64, 64)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="matrix"):
        moe.moe_microscale_dequantize(layer["gate_up_codes"], layer["gate_up_scales"])
    for call in (moe.moe_microscale_product, moe.moe_microscale_gated_product):
        with pytest.raises(ValueError, match="matrix"):
            call(layer["gate_up_codes"], layer["gate_up_scales"], *wt, offsets=off)
        with pytest.raises(ValueError, match="matrix"):
            call(c[0], s[0], *wt, offsets=off)
        for w in (quantised(64), quantised(2, 3, 64, 64)):
            with pytest.raises(ValueError, match="w_codes"):
                call(c, s, *w)
    with pytest.raises(ValueError, match="route_row"):
        moe.moe_microscale_quantize(torch.zeros(3, 64), route_row=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="topk_ids"):
        moe.moe_token_plan(torch.zeros(3, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="topk_ids"):
        h, _, w = step_args()
        moe.moe_microscale_ffn(h, layer, torch.zeros(3, dtype=torch.int32), w)
    assert launches(fake) == []
    moe.moe_microscale_dequantize(c, s)
    moe.moe_microscale_product(c, s, *wt, offsets=off)
    moe.moe_microscale_product(c, s, wt[0][0], wt[1][0])
    assert len(launches(fake)) == 3


def test_tensors_of_a_device_that_is_not_current_are_refused(monkeypatch):
    """The library launches on the current device; the other's default stream has the same
    handle, 0."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    assert moe._raw_stream(None, torch.device("cuda", 0)) == 0
    for stream in (None, 0, 1 << 20):
        with pytest.raises(ValueError, match="current device"):
            moe._raw_stream(stream, torch.device("cuda", 1))


def test_the_current_stream_without_the_raw_handle(monkeypatch):
    """Where torch has no call for the raw handle the public one serves."""
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert moe._raw_stream(None, torch.device("cuda", 0)) == 77
    assert moe._stream(None).value == 77
