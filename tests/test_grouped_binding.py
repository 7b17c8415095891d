"""What the grouped products and checkpoint calls check before anything is launched, on the CPU:
the C entry points with addresses that are never read, the binding over a fake library."""
import ctypes

import pytest
import torch

import __graft_entry__ as entry
from routed_expert_ffn_top_gb300 import moe
from test_tokens_binding import BAD_WORKSPACES, Recorder, fake, launches  # noqa: F401

A = 1 << 20  # an aligned address; never dereferenced by validation
OK, BAD, UNSUPPORTED, SPACE = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return moe.lib()


# ------------------------------------------------------------------------------ C entry points
PRODUCT = dict(x=A, ldx=64, rows=5, dtype=0, offsets=A, w=A, w2=None, transposed=0, E=4, N=96, K=64, y_dtype=0, y=A, ldy=96,
               work=A, bytes=256, stream=None)
GATED = dict(x=A, ldx=64, rows=5, dtype=0, offsets=A, w_gate=A, w_up=A, E=4, I=96, H=64, p=A, ldp=96, code=0, codes=A, scales=A,
             work=A, bytes=256, stream=None)
GRAD = dict(x=A, ldx=64, rows=5, dtype=0, offsets=A, w_down=A, E=4, I=96, H=64, code=0, codes=A, scales=A, out=A, p=A, work=A,
            bytes=256, stream=None)
WEIGHTS = dict(x=A, ldx=64, grads=A, ldg=96, rows=5, dtype=0, offsets=A, E=4, K=64, N=96, out_dtype=2, out=A, work=A, bytes=256,
               stream=None)
CALLS = {"moe_grouped_product": PRODUCT, "moe_grouped_gated_product": GATED, "moe_grouped_gated_product_grad": GRAD,
         "moe_grouped_weight_grad": WEIGHTS}


def result(lib, name, **changed):
    args = dict(CALLS[name], **changed)
    assert len(args) == len(CALLS[name])
    return getattr(lib, name)(*args.values())


COMMON = [(dict(rows=-1), BAD), (dict(E=0), BAD), (dict(dtype=2), BAD), (dict(dtype=7), BAD), (dict(E=1025), UNSUPPORTED),
          (dict(rows=1 << 24), UNSUPPORTED), (dict(offsets=None), BAD), (dict(offsets=A + 2), BAD), (dict(work=None), BAD),
          (dict(work=A + 8), BAD), (dict(bytes=255), SPACE), (dict(x=None), BAD), (dict(x=A + 8), BAD), (dict(ldx=60), BAD),
          (dict(ldx=68), UNSUPPORTED), (dict(ldx=1 << 36), UNSUPPORTED)]


@pytest.mark.parametrize("name", list(CALLS))
def test_common_refusals(lib, name):
    for changed, want in COMMON:
        assert result(lib, name, **changed) == want, changed
    if name != "moe_grouped_weight_grad":
        assert result(lib, name, rows=0, x=None, offsets=A) == OK  # nothing to do


def test_product_refusals(lib):
    for changed, want in [(dict(N=0), BAD), (dict(K=-8), BAD), (dict(N=100), UNSUPPORTED), (dict(K=60, ldx=64), UNSUPPORTED),
                          (dict(N=(1 << 20) + 8), UNSUPPORTED), (dict(w=None), BAD), (dict(w=A + 8), BAD), (dict(w2=A + 4), BAD),
                          (dict(w2=A), BAD),  # rows of 64 columns are not two halves of 64
                          (dict(y_dtype=3), BAD), (dict(y=None), BAD), (dict(y=A + 1), BAD), (dict(y_dtype=2, y=A + 2), BAD),
                          (dict(ldy=95), BAD)]:
        assert result(lib, "moe_grouped_product", **changed) == want, changed


def test_gated_refusals(lib):
    for changed, want in [(dict(I=0), BAD), (dict(I=40, ldp=96), UNSUPPORTED), (dict(H=60), UNSUPPORTED), (dict(I=1 << 20), UNSUPPORTED),
                          (dict(w_gate=None), BAD), (dict(w_up=A + 8), BAD), (dict(codes=None), BAD), (dict(scales=None), BAD),
                          (dict(code=2), BAD), (dict(codes=A + 8), BAD), (dict(scales=A + 8), BAD), (dict(p=None), BAD),
                          (dict(p=A + 1), BAD), (dict(ldp=95), BAD)]:
        assert result(lib, "moe_grouped_gated_product", **changed) == want, changed


def test_gated_grad_refusals(lib):
    for changed, want in [(dict(I=40), UNSUPPORTED), (dict(H=60), UNSUPPORTED), (dict(code=-1), BAD), (dict(w_down=None), BAD),
                          (dict(codes=None), BAD), (dict(codes=A + 8), BAD), (dict(scales=None), BAD), (dict(out=None), BAD),
                          (dict(out=A + 8), BAD), (dict(p=A + 8), BAD)]:
        assert result(lib, "moe_grouped_gated_product_grad", **changed) == want, changed


def test_weight_grad_refusals(lib):
    for changed, want in [(dict(K=60), UNSUPPORTED), (dict(N=92), UNSUPPORTED), (dict(grads=None), BAD), (dict(grads=A + 8), BAD),
                          (dict(ldg=88), BAD), (dict(ldg=100), UNSUPPORTED), (dict(out_dtype=3), BAD), (dict(out=None), BAD),
                          (dict(out=A + 8), BAD), (dict(E=1024, K=1 << 20, N=1 << 20, ldx=1 << 20, ldg=1 << 20), UNSUPPORTED)]:
        assert result(lib, "moe_grouped_weight_grad", **changed) == want, changed


def test_checkpoint_refusals(lib):
    quantize = dict(x=A, ldx=64, dtype=0, rows=3, cols=64, code=0, codes=A, scales=A, stream=None)
    for changed, want in [(dict(rows=-1), BAD), (dict(dtype=3), BAD), (dict(code=2), BAD), (dict(cols=0), BAD), (dict(cols=48), UNSUPPORTED),
                          (dict(cols=(1 << 20) + 32), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(x=None), BAD), (dict(x=A + 1), BAD),
                          (dict(ldx=32), BAD), (dict(codes=None), BAD), (dict(codes=A + 8), BAD), (dict(scales=A + 8), BAD), (dict(rows=0, x=None), OK)]:
        assert lib.moe_checkpoint_quantize(*dict(quantize, **changed).values()) == want, changed
    back = dict(codes=A, scales=A, code=1, rows=3, cols=64, rr=A, k=2, x=A, ldx=64, dtype=0, stream=None)
    for changed, want in [(dict(rows=-1), BAD), (dict(dtype=3), BAD), (dict(code=2), BAD), (dict(cols=48), UNSUPPORTED), (dict(k=0), BAD),
                          (dict(k=33), UNSUPPORTED), (dict(rows=1 << 23, k=2), UNSUPPORTED), (dict(rr=A + 2), BAD), (dict(x=None), BAD),
                          (dict(ldx=63), BAD), (dict(codes=None), BAD), (dict(scales=A + 4), BAD), (dict(rows=0, codes=None), OK)]:
        assert lib.moe_checkpoint_dequantize(*dict(back, **changed).values()) == want, changed
    assert [lib.moe_checkpoint_pitch(c) for c in (32, 512, 544, 0, 33, (1 << 20) + 32)] == [16, 16, 32, 0, 0, 0]


# ------------------------------------------------------------------------------------ binding
def tensors(R=6, E=3, H=64, I=32, dtype=BF16, device="cpu"):
    def z(*shape, dt=dtype):
        return torch.zeros(shape, dtype=dt, device=device)
    return {"rows": z(R, H), "gate": z(E, H, I), "up": z(E, H, I), "down": z(E, I, H), "off": z(E + 1, dt=torch.int32), "gy": z(R, H),
            "codes": z(R, 2 * I, dt=torch.int8), "scales": z(R, 16, dt=torch.uint8), "p": z(R, I), "work": z(256, dt=torch.uint8)}


def calls(t, **kw):
    kw = dict({"workspace": t["work"]}, **kw)
    return [lambda: moe.moe_grouped_product(t["rows"], t["gate"], t["off"], **kw),
            lambda: moe.moe_grouped_product(torch.cat((t["p"], t["p"]), 1), (t["gate"], t["up"]), t["off"], transposed=True, **kw),
            lambda: moe.moe_grouped_gated_product(t["rows"], t["gate"], t["up"], t["off"], checkpoint=torch.int8, **kw),
            lambda: moe.moe_grouped_gated_product_grad(t["gy"], t["down"], t["off"], t["codes"], t["scales"], **kw),
            lambda: moe.moe_grouped_weight_grad(t["rows"], t["p"], t["off"], **kw)]


def test_shapes_that_come_back(fake):
    t = tensors()
    y, dx, (p, codes, scales), (ggu, again), gw = [c() for c in calls(t)]
    assert y.shape == (6, 32) and dx.shape == (6, 64) and p.shape == again.shape == (6, 32) and ggu.shape == (6, 64)
    assert codes.shape == (6, 64) and codes.dtype is torch.int8 and scales.shape == (6, 16) and gw.shape == (3, 64, 32)
    assert gw.dtype is F32 and y.dtype is BF16
    assert len(launches(fake)) == 5
    names = [n for n in launches(fake)]
    assert names == ["moe_grouped_product"] * 2 + ["moe_grouped_gated_product", "moe_grouped_gated_product_grad", "moe_grouped_weight_grad"]
    args = dict(zip(PRODUCT, fake.calls[1][1]))  # the pair: K of one half, N the transposes' columns
    assert (args["K"], args["N"], args["ldx"], args["transposed"], args["E"]) == (32, 64, 64, 1, 3)
    assert (args["w"], args["w2"]) == (t["gate"].data_ptr(), t["up"].data_ptr())


def test_types_and_shapes_that_do_not_fit(fake):
    t = tensors()
    z = torch.zeros
    for error, call in [
            (TypeError, lambda: moe.moe_grouped_product(t["rows"].float(), t["gate"].float(), t["off"])),
            (TypeError, lambda: moe.moe_grouped_product(t["rows"], t["gate"].to(F16), t["off"])),
            (TypeError, lambda: moe.moe_grouped_product(t["rows"], t["gate"], t["off"].long())),
            (TypeError, lambda: moe.moe_grouped_product(t["rows"], t["gate"], t["off"], dtype=torch.float64)),
            (TypeError, lambda: moe.moe_grouped_product(t["rows"], t["gate"], t["off"], dtype=F32, out=z(6, 32, dtype=BF16))),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"], t["gate"], t["off"][:-1])),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"], t["gate"], t["off"], transposed=True)),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"], (t["gate"], t["up"]), t["off"])),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"], (t["gate"],) * 3, t["off"])),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"], (t["gate"], t["down"]), t["off"], transposed=True)),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"], t["gate"][:, :, ::2], t["off"])),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"][0], t["gate"], t["off"])),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"], t["gate"].reshape(-1), t["off"])),
            (ValueError, lambda: moe.moe_grouped_product(t["rows"], t["gate"], t["off"], out=z(6, 33, dtype=BF16))),
            (ValueError, lambda: moe.moe_grouped_gated_product(t["rows"], t["gate"], t["down"], t["off"])),
            (ValueError, lambda: moe.moe_grouped_gated_product(t["rows"], t["down"], t["down"], t["off"])),
            (TypeError, lambda: moe.moe_grouped_gated_product(t["rows"], t["gate"], t["up"], t["off"], checkpoint=BF16)),
            (ValueError, lambda: moe.moe_grouped_gated_product(t["rows"], t["gate"], t["up"], t["off"], codes=t["codes"])),
            (TypeError, lambda: moe.moe_grouped_gated_product(t["rows"], t["gate"], t["up"], t["off"], checkpoint=torch.float8_e4m3fn, codes=t["codes"])),
            (ValueError, lambda: moe.moe_grouped_gated_product_grad(t["gy"], t["gate"], t["off"], t["codes"], t["scales"])),
            (ValueError, lambda: moe.moe_grouped_gated_product_grad(t["gy"], t["down"], t["off"], t["codes"][:5], t["scales"][:5])),
            (ValueError, lambda: moe.moe_grouped_gated_product_grad(t["gy"], t["down"], t["off"], t["codes"], t["scales"][:, :8])),
            (TypeError, lambda: moe.moe_grouped_gated_product_grad(t["gy"], t["down"], t["off"], t["codes"].to(torch.uint8), t["scales"])),
            (ValueError, lambda: moe.moe_grouped_weight_grad(t["rows"], t["p"][:5], t["off"])),
            (TypeError, lambda: moe.moe_grouped_weight_grad(t["rows"], t["p"].to(F16), t["off"])),
            (ValueError, lambda: moe.moe_grouped_weight_grad(t["rows"], t["p"], t["off"][:1])),
            (ValueError, lambda: moe.moe_grouped_weight_grad(t["rows"], t["p"], t["off"], out=z(3, 64, 33))),
            (TypeError, lambda: moe.moe_grouped_weight_grad(t["rows"], t["p"], t["off"], dtype=torch.int32)),
            (moe.MoeError, lambda: moe.moe_grouped_gated_product(t["rows"], z(3, 64, 40, dtype=BF16), z(3, 64, 40, dtype=BF16), t["off"])),
            (moe.MoeError, lambda: moe.moe_checkpoint_quantize(z(3, 48))),
            (TypeError, lambda: moe.moe_checkpoint_quantize(z(3, 64), dtype=torch.uint8)),
            (TypeError, lambda: moe.moe_checkpoint_quantize(z(3, 64, dtype=torch.float64))),
            (ValueError, lambda: moe.moe_checkpoint_quantize(z(3, 64), codes=z(3, 32, dtype=torch.float8_e4m3fn))),
            (TypeError, lambda: moe.moe_checkpoint_dequantize(t["codes"], t["scales"], dtype=torch.int32)),
            (ValueError, lambda: moe.moe_checkpoint_dequantize(t["codes"], t["scales"], route_row=z(6, dtype=torch.int32))),
            (ValueError, lambda: moe.moe_checkpoint_dequantize(t["codes"], t["scales"], route_row=z(5, 2, dtype=torch.int32))),
            (ValueError, lambda: moe.moe_checkpoint_dequantize(t["codes"], t["scales"], out=z(6, 32)))]:
        with pytest.raises(error):
            call()
    assert [n for n in launches(fake) if n != "moe_status_string"] == []  # (an error's own text)


def test_tensors_of_one_device(fake):
    for name in ("gate", "up", "down", "off", "codes", "scales", "p"):
        t = tensors()
        t[name] = t[name].to("meta")
        failed = 0
        for call in calls(t):
            try:
                call()
            except ValueError as e:
                assert "meta" in str(e)
                failed += 1
            except (RuntimeError, NotImplementedError):  # torch's own: the pair's rows are joined before the call
                failed += 1
        assert failed > 0
        for _, args in fake.calls:
            assert None not in args[:1]


@pytest.mark.parametrize("work,error", BAD_WORKSPACES)
def test_a_workspace_is_contiguous_bytes_of_the_device(fake, work, error):
    for call in calls(tensors(), workspace=work):
        with pytest.raises(error):
            call()
    assert launches(fake) == []


@pytest.mark.parametrize("capturing", [False, True])
def test_a_call_without_a_workspace_reports_what_the_device_found(fake, monkeypatch, capturing):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    for call in calls(tensors(), workspace=None):
        fake.calls.clear()
        call()
        assert launches(fake).count("moe_read_device_status") == (0 if capturing else 1)
    if capturing:
        return

    def status(*args):
        ctypes.cast(args[2], ctypes.POINTER(ctypes.c_int32))[0] = moe.MOE_DEV_WAIT_TIMEOUT
        return moe.MOE_ERR_DEVICE
    fake.moe_read_device_status = status
    for call in calls(tensors(), workspace=None):
        with pytest.raises(moe.MoeError):
            call()


def test_allocations_are_the_launch_streams(fake, monkeypatch):
    """What a call allocates belongs to the stream that it launches on."""
    depth, seen = [0], []

    class On:
        def __enter__(self):
            depth[0] += 1

        def __exit__(self, *_):
            depth[0] -= 1
    t = tensors()
    x = torch.zeros(6, 64)
    rr = torch.zeros((6, 2), dtype=torch.int32)
    some = calls(t, stream=5, workspace=None) + [
        lambda: moe.moe_checkpoint_quantize(x, stream=5), lambda: moe.moe_checkpoint_dequantize(t["codes"], t["scales"], stream=5),
        lambda: moe.moe_checkpoint_dequantize(t["codes"], t["scales"], route_row=rr, stream=5)]
    monkeypatch.setattr(moe, "_launch_stream", lambda stream, device: On())
    monkeypatch.setattr(moe, "_check", lambda rc, where: seen.append((where, depth[0])))
    for name in ("empty", "zeros"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, real=real, name=name, **kw: seen.append((name, depth[0])) or real(*a, **kw))
    for call in some:
        seen.clear()
        call()
        assert len(seen) > 1 and all(d == 1 for _, d in seen), seen


def test_tensors_of_a_device_that_is_not_current_are_refused(fake, monkeypatch):
    def refuse(device):
        raise ValueError("current device")
    monkeypatch.setattr(moe, "_raw_stream", refuse)
    t = tensors()
    for call in calls(t) + [lambda: moe.moe_checkpoint_quantize(t["rows"]), lambda: moe.moe_checkpoint_dequantize(t["codes"], t["scales"])]:
        with pytest.raises(ValueError, match="current device"):
            call()
    assert launches(fake) == []
