"""What the Python binding of the calls for many tokens refuses, and what it
passes on, seen without a GPU: tensors that say they are on one, and a
stand-in for the library that records the calls."""
import pytest
import torch

import mxfp4_weight_streaming_gb300 as mx
from mxfp4_weight_streaming_gb300 import step
from test_step_binding import Library, OnGpu

BF16, E4M3, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8


@pytest.fixture(autouse=True)
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(step, "_L", lib)
    monkeypatch.setattr(step, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(step, "_current_device", lambda: 0, raising=False)
    return lib


def make(*shape, dtype=BF16, device=0):
    t = torch.zeros(shape, dtype=U8 if dtype == E4M3 else dtype)
    return OnGpu(t.view(E4M3) if dtype == E4M3 else t, device)


def codes(t, k, form="e4m3", device=0):
    return (make(t, k, dtype=E4M3, device=device) if form == "e4m3" else make(t, k // 2, dtype=U8, device=device),
            make(t, k // 32, dtype=U8, device=device))


@pytest.mark.parametrize("form,number", [("e4m3", 0), ("e2m1", 1)])
def test_linear_passes_its_sizes(library, form, number):
    x, w = codes(5, 256, form), codes(7, 256, "e2m1")
    y = make(5, 7)
    assert mx.linear_mx(*x, *w, out=y) is y
    name, args = library.calls[-1]
    assert name == "mxfp4_linear_mx" and args[2:5] == (number, 5, 256) and args[7] == 7
    assert args[0] == x[0].data_ptr() and args[8] == y.data_ptr()


def test_swiglu_and_quantize_pass_their_sizes(library):
    out = codes(5, 96, "e2m1")
    assert mx.swiglu_mx(*codes(5, 256), *codes(192, 256, "e2m1"), format="e2m1", out=out) == out
    name, args = library.calls[-1]
    assert name == "mxfp4_swiglu_mx" and args[2:5] == (0, 5, 256) and args[7:9] == (96, 1)
    wide = torch.zeros(6, 640, dtype=BF16)
    mx.quantize_mx(OnGpu(wide[:, 64:576]), out=codes(6, 512))
    assert library.calls[-1][1][1:6] == (640, 6, 512, 0, 0)
    mx.quantize_mx(OnGpu(wide[:, 64:576]), "e2m1", swiglu=True, out=codes(6, 256, "e2m1"))
    assert library.calls[-1][1][1:6] == (640, 6, 256, 1, 1)
    mx.quantize_mx(OnGpu(wide[:1, :512].expand(1, 512)), out=codes(1, 512))
    assert library.calls[-1][1][1] == 512  # one row's stride says nothing


def test_norm_passes_its_arguments(library):
    out, r = codes(3, 64), make(3, 64)
    mx.residual_norm_mx(make(3, 64), make(3, 64), make(64), gate=OnGpu(torch.zeros(3, 128, dtype=BF16)[:, :64]), scale=0.5,
                        kind="layer", out=out, residual_out=r)
    name, args = library.calls[-1]
    assert name == "mxfp4_residual_norm_mx" and args[2:4] == (3, 64) and args[7:9] == (128, 0.5) and args[13:15] == (True, 0)
    assert args[15:18] == (out[0].data_ptr(), out[1].data_ptr(), r.data_ptr())


@pytest.mark.parametrize("what", [
    lambda: mx.linear_mx(make(5, 256), *codes(5, 256)[1:], *codes(7, 256, "e2m1")),                # bf16 activations
    lambda: mx.linear_mx(*codes(5, 256), *codes(7, 128, "e2m1")),                                  # another k
    lambda: mx.linear_mx(codes(5, 256)[0], codes(4, 256)[1], *codes(7, 256, "e2m1")),              # another t
    lambda: mx.linear_mx(*codes(5, 256), codes(7, 256, "e2m1")[0], codes(8, 256)[1]),
    lambda: mx.linear_mx(*codes(5, 256), *codes(7, 256)),                                          # 8-bit weights
    lambda: mx.linear_mx(*codes(5, 256), *codes(7, 256, "e2m1"), out=make(5, 8)),
    lambda: mx.linear_mx(*codes(5, 256), *codes(7, 256, "e2m1"), out=make(5, 7, dtype=torch.float32)),
    lambda: mx.linear_mx(*codes(5, 256), *codes(7, 256, "e2m1"), out=make(5, 7, device=1)),
    lambda: mx.linear_mx(*codes(5, 256, device=1), *codes(7, 256, "e2m1")),
    lambda: mx.linear_mx(*codes(5, 256), *codes(7, 256, "e2m1", device=1)),
    lambda: mx.linear_mx(*codes(5, 256, device=-1), *codes(7, 256, "e2m1", device=-1)),
    lambda: mx.linear_mx(OnGpu(codes(5, 512)[0].t[:, :256]), codes(5, 256)[1], *codes(7, 256, "e2m1")),  # strided rows
    lambda: mx.swiglu_mx(*codes(5, 256), *codes(7, 256, "e2m1")),                                  # an odd number of rows
    lambda: mx.swiglu_mx(*codes(5, 256), *codes(96, 256, "e2m1")),                                 # inter 48
    lambda: mx.swiglu_mx(*codes(5, 256), *codes(64, 256, "e2m1"), format="int8"),
    lambda: mx.swiglu_mx(*codes(5, 256), *codes(64, 256, "e2m1"), out=codes(5, 32, "e2m1")),       # out of another type
    lambda: mx.quantize_mx(make(3, 64, dtype=torch.float32)),
    lambda: mx.quantize_mx(make(64)),
    lambda: mx.quantize_mx(make(3, 64, device=1)),
    lambda: mx.quantize_mx(OnGpu(torch.zeros(64, 3, dtype=BF16).t())),
    lambda: mx.quantize_mx(OnGpu(torch.zeros(1, 64, dtype=BF16).expand(3, 64))),
    lambda: mx.quantize_mx(make(3, 63), swiglu=True),
    lambda: mx.quantize_mx(make(3, 64), "e5m2"),
    lambda: mx.quantize_mx(make(3, 64), out=codes(3, 32)),
    lambda: mx.quantize_mx(make(3, 64), out=(codes(3, 64)[0], codes(3, 64, device=1)[1])),
    lambda: mx.residual_norm_mx(make(3, 64), make(3, 64), make(64), format="bf16"),
    lambda: mx.residual_norm_mx(make(3, 64), make(3, 64), make(64), kind="batch", out=codes(3, 64)),
    lambda: mx.residual_norm_mx(make(3, 64), make(4, 64), make(64), out=codes(3, 64)),
    lambda: mx.residual_norm_mx(make(3, 64), make(3, 64), make(64), out=codes(3, 64), residual_out=make(3, 32)),
    lambda: mx.residual_norm_mx(make(3, 64), make(3, 64), make(64, device=1), out=codes(3, 64)),
    lambda: mx.residual_norm_mx(make(3, 64), make(3, 64), make(64), out=codes(3, 64, device=1))])
def test_refusals(library, what):
    with pytest.raises(ValueError):
        what()
    assert not library.calls
