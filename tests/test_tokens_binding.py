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
            return 4096 if name.endswith("_bytes") else b"status" if name == "moe_status_string" else moe.MOE_OK
        return call


@pytest.fixture
def fake(monkeypatch):
    """The binding with host tensors in the place of the GPU's and the library recorded."""
    r = Recorder()
    monkeypatch.setattr(moe, "lib", lambda: r)
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
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
    assert len([n for n in launches(fake) if n != "moe_read_device_status"]) == 3


def test_tensors_of_a_device_that_is_not_current_are_refused(monkeypatch):
    """The library launches on the current device; the other's default stream has the same
    handle, 0."""
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    monkeypatch.setattr(moe, "_current_stream", lambda index: 0)
    assert moe._raw_stream(torch.device("cuda", 0)) == 0
    with pytest.raises(ValueError, match="current device"):
        moe._raw_stream(torch.device("cuda", 1))


def test_the_current_stream_without_the_raw_handle(lib, monkeypatch):
    """Where torch has no call for the raw handle the public one serves."""
    import importlib.util

    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("routed_expert_ffn_top_gb300.moe_again", moe.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._raw_stream(torch.device("cuda", 0)) == 77
    assert again._stream(None).value == 77


def calls_with_stream(stream):
    """Every call that allocates, given a stream."""
    h, ids, w = step_args()
    layer, (c, s), wt = four_bit_layer(), quantised(3, 64), quantised(2, 64, 64)
    off = torch.zeros(3, dtype=torch.int32)
    x, rows = torch.zeros(3, 64), torch.zeros(6, 64)
    dense = {"H": 64, "I": 32, "E": 2, "w_gate": torch.zeros(2, 64, 32), "w_up": torch.zeros(2, 64, 32),
             "w_down": torch.zeros(2, 32, 64)}
    return [lambda: moe.moe_token_plan(ids, 4, stream=stream), lambda: moe.moe_token_sort(x, ids, stream=stream),
            lambda: moe.moe_token_sort_grad(rows, ids, stream=stream),
            lambda: moe.moe_token_unsort(rows, ids, w, residual=x, stream=stream),
            lambda: moe.moe_token_unsort_grad(x, rows, ids, w, stream=stream),
            lambda: moe.moe_microscale_quantize(x, stream=stream),
            lambda: moe.moe_microscale_quantize(x, route_row=ids, stream=stream),
            lambda: moe.moe_microscale_dequantize(c, s, stream=stream),
            lambda: moe.moe_microscale_product(c, s, *wt, offsets=off, stream=stream),
            lambda: moe.moe_microscale_gated_product(c, s, *wt, offsets=off, stream=stream),
            lambda: moe.microscale_layer(dense, stream=stream),
            lambda: moe.moe_microscale_ffn(h, layer, ids, w, residual=h, stream=stream)]


@pytest.mark.parametrize("i", range(12))
def test_allocations_are_the_launch_streams(fake, monkeypatch, i):
    """What a call allocates, fills or copies itself belongs to the stream that it launches on:
    memory of another stream may still be in use there, and is given away there too soon."""
    depth, seen = [0], []

    class On:
        def __enter__(self):
            depth[0] += 1

        def __exit__(self, *_):
            depth[0] -= 1

    def watch(owner, name):
        real = getattr(owner, name)

        def call(*args, **kw):
            seen.append((name, depth[0]))
            return real(*args, **kw)
        monkeypatch.setattr(owner, name, call)

    call = calls_with_stream(5)[i]
    monkeypatch.setattr(moe, "_launch_stream", lambda stream, device: On(), raising=False)
    monkeypatch.setattr(moe, "_check", lambda rc, where: seen.append((where, depth[0])))
    for owner, name in ((torch, "empty"), (torch, "zeros"), (torch.Tensor, "contiguous")):
        watch(owner, name)
    call()
    assert len(seen) > 1 and all(d == 1 for _, d in seen), seen


def test_a_stream_is_taken_as_an_object_or_a_handle(monkeypatch):
    class Stream:
        def __init__(self, handle, device=None):
            self.handle, self.device = handle, device
    cuda = torch.device("cuda", 0)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream("default", device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    mine = Stream(3)
    assert moe._launch_stream(mine, cuda) is mine
    assert moe._launch_stream(1 << 20, cuda).handle == 1 << 20
    assert moe._launch_stream(0, cuda).handle == "default"
    with pytest.raises(ValueError):
        moe._launch_stream(mine, torch.device("cpu"))


@pytest.mark.parametrize("capturing", [False, True])
def test_a_call_without_a_workspace_reports_what_the_device_found(fake, monkeypatch, capturing):
    """Its status word has no other reader: the call waits and raises.  A call that is being
    captured in a graph cannot wait."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    h, ids, w = step_args()
    layer, x, wt = four_bit_layer(), quantised(3, 64), quantised(2, 64, 64)
    off = torch.zeros(3, dtype=torch.int32)
    work = torch.zeros(8192, dtype=torch.uint8)
    calls = [lambda ws: moe.moe_microscale_product(*x, *wt, offsets=off, workspace=ws),
             lambda ws: moe.moe_microscale_gated_product(*x, *wt, offsets=off, workspace=ws),
             lambda ws: moe.moe_microscale_ffn(h, layer, ids, w, workspace=ws)]
    for call in calls:
        fake.calls.clear()
        call(work)
        assert "moe_read_device_status" not in launches(fake)
        call(None)
        assert launches(fake).count("moe_read_device_status") == (0 if capturing else 1)
    if capturing:
        return

    def status(*args):
        ctypes.cast(args[2], ctypes.POINTER(ctypes.c_int32))[0] = moe.MOE_DEV_WAIT_TIMEOUT
        return moe.MOE_ERR_DEVICE
    fake.moe_read_device_status = status
    for call in calls:
        call(work)
        with pytest.raises(moe.MoeError):
            call(None)


def test_a_new_workspace_is_filled_where_it_must_be(monkeypatch):
    """Only the status word has to be zero; a prompt's workspace is hundreds of megabytes."""
    layer = {k: v.to("meta") if isinstance(v, torch.Tensor) else v for k, v in four_bit_layer(H=2048, I=768).items()}
    filled = []
    real = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: filled.append(real(*a, **kw)) or filled[-1])
    zero_ = torch.Tensor.zero_
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: filled.append(t) or zero_(t))
    monkeypatch.setattr(moe, "lib", Recorder)
    monkeypatch.setattr(moe, "moe_microscale_workspace_bytes", lambda *a: 1 << 28)
    work = moe.microscale_workspace(layer, 8192, 8)
    assert work.numel() == 1 << 28 and work.dtype is torch.uint8
    assert sum(t.numel() for t in filled) == moe.MOE_MICROSCALE_STATUS_BYTES


def test_status_read_refuses(lib):
    out = ctypes.c_int32(0)
    for work, result in ((None, ctypes.byref(out)), (A + 8, ctypes.byref(out)), (A, None)):
        assert lib.moe_read_device_status(work, None, result) == moe.MOE_ERR_INVALID_ARG


def test_type_of_the_rows_before_their_sum(lib, fake):
    layer = four_bit_layer()
    assert moe.microscale_weights(layer).y_dtype == moe.MOE_DT_BF16
    layer["y_dtype"] = torch.float32
    assert moe.microscale_weights(layer).y_dtype == moe.MOE_DT_F32
    layer["y_dtype"] = torch.float16
    with pytest.raises(TypeError):
        moe.microscale_weights(layer)

    def need(y):
        return lib.moe_microscale_workspace_bytes(ctypes.byref(moe.MicroscaleWeights(64, 32, 4, y, A, A, A, A)), 40, 2)
    assert need(moe.MOE_DT_F32) == need(moe.MOE_DT_BF16) + 80 * 64 * 2
    for y in (moe.MOE_DT_F16, 3, -1):
        w = moe.MicroscaleWeights(64, 32, 4, y, A, A, A, A)
        assert need(y) == 0
        assert lib.moe_microscale_ffn(A, ctypes.byref(w), 4, 2, A, A, None, A, A, 1 << 30, None) == moe.MOE_ERR_INVALID_ARG


def dense_layer(E=4, H=64, I=32, device="cpu"):
    bf16 = torch.bfloat16
    return {"H": H, "I": I, "E": E, "w_gate": torch.zeros((E, H, I), dtype=bf16, device=device),
            "w_up": torch.zeros((E, H, I), dtype=bf16, device=device), "w_down": torch.zeros((E, I, H), dtype=bf16, device=device),
            "w_router": torch.zeros((H, E), dtype=bf16, device=device), "bias": None}


@pytest.fixture
def posing(fake, monkeypatch):
    """Host tensors in the place of the GPU's for the block's calls too."""
    monkeypatch.setattr(moe, "_stream", lambda stream: None)
    monkeypatch.setattr(moe, "_need_cuda", lambda device: None)
    return fake


def block_calls(h, ids, w, work):
    return [lambda layer: moe.moe_expert_ffn(h, layer, ids, w, 8, workspace=work),
            lambda layer: moe.moe_decode_block(h, layer, 2, 8, workspace=work),
            lambda layer: moe.moe_decode_block_noalloc(h, layer, 2, 8)]


def test_block_takes_a_layer_of_its_own_device_only(posing):
    h, ids, w = step_args()
    for call in block_calls(h, ids, w, torch.zeros(8192, dtype=torch.uint8)):
        call(dense_layer())
        assert len(launches(posing)) == 1
        posing.calls.clear()
        layer = dense_layer(device="meta")
        layer["w_router"] = torch.zeros((64, 4), dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="meta"):
            call(layer)
        assert launches(posing) == []


@pytest.mark.parametrize("work,error", BAD_WORKSPACES)
def test_a_blocks_workspace_is_contiguous_bytes_of_the_device(posing, work, error):
    h, ids, w = step_args()
    for call in block_calls(h, ids, w, work)[:2]:
        with pytest.raises(error):
            call(dense_layer())
    rd = {"H": 64, "I": 32, "E": 4, "rank": 4}
    for name in ("signs", "g_rows", "v_rows", "w_down", "g_codes", "v_codes", "g_scales", "v_scales", "dnorm", "U", "coef"):
        rd[name] = torch.zeros(64)
    with pytest.raises(error):
        moe.moe_reader_ffn(h, rd, ids, w, 8, workspace=work)
    assert launches(posing) == []


def test_block_refuses_host_tensors(fake, monkeypatch):
    monkeypatch.setattr(moe, "_stream", lambda stream: None)
    h, ids, w = step_args()
    work = torch.zeros(8192, dtype=torch.uint8)
    for call in block_calls(h, ids, w, work):
        with pytest.raises(ValueError, match="CUDA"):
            call(dense_layer())
    for call in (lambda: moe.moe_route_topk(h, dense_layer()["w_router"], None, 2),
                 lambda: moe.moe_align_block_size(ids, 4, 8),
                 lambda: moe.moe_reader_ffn(h, {"w_down": h}, ids, w, 8, workspace=work)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert launches(fake) == []
