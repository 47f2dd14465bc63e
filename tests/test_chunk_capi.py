"""Argument checks of the entry points for many tokens: every refusal comes
before any launch (these calls need no GPU)."""
import pytest

import mxfp4_weight_streaming_gb300 as mx

A, B, C, D, E, F = (0x10000000 * (i + 1) for i in range(6))  # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mxfp4_weight_streaming_gb300 import build
    build.build()
    return mx.load()


def call(f, base, change):
    a = dict(base, **change)
    return getattr(mx.load(), f)(*a.values())


QUANTIZE = dict(x=A, x_stride=0, t=4, k=256, swiglu=0, format=0, xq=B, xs=C, stream=None)
NORM = dict(x=A, residual=B, tokens=4, n=256, post_weight=None, post_bias=None, gate=None, gate_stride=0, scale=1.0,
            weight=C, bias=None, weight_offset=0.0, eps=1e-6, layer=0, format=0, yq=D, ys=E, r_out=F, stream=None)
LINEAR = dict(xq=A, xs=B, format=0, t=4, k=256, wq=C, ws=D, n=100, y=E, stream=None)
SWIGLU = dict(xq=A, xs=B, format=0, t=4, k=256, w1q=C, w1s=D, inter=96, out_format=1, hq=E, hs=F, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(xq=None), 1), (dict(xs=None), 1), (dict(t=0), 1), (dict(t=-1), 1), (dict(k=0), 1),
    (dict(format=2), 1), (dict(format=-1), 1), (dict(x_stride=248), 1), (dict(x_stride=-8), 1),
    (dict(swiglu=1, x_stride=504), 1), (dict(k=250), 2), (dict(k=1 << 31), 2), (dict(t=1 << 31), 2),
    (dict(x_stride=1 << 31), 2), (dict(x=A + 8), 3), (dict(x_stride=260), 3), (dict(xq=B + 8), 3),
    # outputs in the input, or in each other
    (dict(xq=A), 1), (dict(xq=A + 4 * 512 - 16), 1), (dict(xs=A + 100), 1), (dict(xs=B + 4 * 256 - 1), 1),
    (dict(x_stride=512, xq=A + 3 * 1024 + 496), 1)])
def test_quantize_refusals(change, status):
    assert call("mxfp4_quantize_mx", QUANTIZE, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(residual=None), 1), (dict(weight=None), 1), (dict(yq=None), 1), (dict(ys=None), 1),
    (dict(r_out=None), 1), (dict(tokens=0), 1), (dict(n=0), 1), (dict(post_bias=C), 1), (dict(gate_stride=-8), 1),
    (dict(gate=C, gate_stride=248), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(format=2), 1),
    (dict(n=32768 + 32), 2), (dict(n=248), 2), (dict(tokens=1 << 31), 2), (dict(gate=C, gate_stride=1 << 31), 2),
    (dict(x=A + 2), 3), (dict(residual=B + 8), 3), (dict(weight=C + 4), 3), (dict(yq=D + 8), 3), (dict(r_out=F + 2), 3),
    (dict(gate=C + 2), 3), (dict(gate=C, gate_stride=260), 3), (dict(yq=A), 1), (dict(yq=B + 16), 1), (dict(yq=F), 1),
    (dict(ys=A), 1), (dict(ys=D + 1023), 1), (dict(yq=C), 1)])
def test_norm_refusals(change, status):
    assert call("mxfp4_residual_norm_mx", NORM, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(xq=None), 1), (dict(xs=None), 1), (dict(wq=None), 1), (dict(ws=None), 1), (dict(y=None), 1), (dict(t=0), 1),
    (dict(k=0), 1), (dict(n=0), 1), (dict(format=2), 1), (dict(k=192), 2), (dict(k=32), 2), (dict(t=1 << 31), 2),
    (dict(n=1 << 31), 2), (dict(k=1 << 31), 2), (dict(k=(1 << 24) + 128), 2), (dict(xq=A + 8), 3), (dict(xs=B + 2), 3), (dict(ws=D + 1), 3),
    (dict(wq=C + 16), 3), (dict(wq=C + 8, format=1), 3), (dict(y=E + 1), 3),
    (dict(y=A), 1), (dict(y=B + 4 * 8 - 2), 1), (dict(y=C - 2), 1), (dict(y=D), 1)])
def test_linear_refusals(change, status):
    assert call("mxfp4_linear_mx", LINEAR, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(xq=None), 1), (dict(w1q=None), 1), (dict(hq=None), 1), (dict(hs=None), 1), (dict(inter=0), 1),
    (dict(out_format=2), 1), (dict(out_format=-1), 1), (dict(inter=80), 2), (dict(inter=1 << 30), 2), (dict(k=64), 2),
    (dict(hq=E + 8), 3), (dict(hq=A), 1), (dict(hs=E), 1), (dict(hs=D + 2 * 96 * 8 - 1), 1)])
def test_swiglu_refusals(change, status):
    assert call("mxfp4_swiglu_mx", SWIGLU, change) == status


@pytest.mark.parametrize("change", [
    dict(r_out=C), dict(r_out=C + 496), dict(bias=F, r_out=F), dict(post_weight=F + 2032, r_out=F),
    dict(post_weight=A, post_bias=F, r_out=F), dict(gate=F, r_out=F), dict(gate=F, gate_stride=256, r_out=F),
    dict(gate=F - 3 * 1024 - 496, gate_stride=512, r_out=F), dict(r_out=A + 512), dict(r_out=A - 16), dict(r_out=B + 512),
    dict(r_out=B - 2032)])
def test_norm_refuses_a_sum_over_its_inputs(change):
    """r over a vector that every row reads, over the gates, or over x or the residual a few rows on."""
    assert call("mxfp4_residual_norm_mx", NORM, change) == 1
