"""Many tokens at once (prompt chunks, large batches) over the C ABI:
activations as microscaled (MX) codes, and their products with MXFP4 weights
(include/mxfp4.h has the definitions). Argument marshalling only, as in the
rest of the binding.

MX codes of [t, k] activations are a pair of tensors: float8_e4m3fn [t, k] or
uint8 [t, k / 2] (E2M1, two a byte), and uint8 scales [t, k / 32]. All tensors
of a call lie on the current GPU. With stream= a call runs on that stream, and
the results it makes are that stream's memory.
"""
from __future__ import annotations

import torch

from . import step
from .step import _BF16, _E4M3, _fail, _lib, _made, _need, _on_device, _ptr, _stream_of, _strides

_U8 = torch.uint8
_FORMATS = {"e4m3": 0, "e2m1": 1}


def _format(name):
    number = _FORMATS.get(name)
    if number is None:
        raise ValueError("format: 'e4m3' or 'e2m1' expected")
    return number


def _raw(stream, device, *given):
    return step._raw_stream(device) if stream is None else _stream_of(stream, *given)


def _outputs(out, number, t, k, device, stream):
    """(codes, scales) for t rows of k values: the caller's, or new ones."""
    dtype, width = (_E4M3, k) if number == 0 else (_U8, k // 2)
    if out is None:
        return _made(stream, (t, width), dtype, device), _made(stream, (t, k // 32), _U8, device)
    q, s = out
    if q.dtype is not dtype or q.shape != (t, width) or not q.is_contiguous() or s.dtype is not _U8 or \
            s.shape != (t, k // 32) or not s.is_contiguous():
        raise ValueError("out: contiguous codes (float8_e4m3fn [t, k] or uint8 [t, k / 2]) and uint8 scales [t, k / 32] expected")
    return q, s


def _codes(q, s):
    """(format, t, k) of activations as the products take them."""
    if q.dtype is _E4M3 and q.dim() == 2:
        number, t, k = 0, q.shape[0], q.shape[1]
    elif q.dtype is _U8 and q.dim() == 2:
        number, t, k = 1, q.shape[0], 2 * q.shape[1]
    else:
        raise ValueError("xq: float8_e4m3fn [t, k] or uint8 [t, k / 2] expected")
    if not q.is_cuda or not q.is_contiguous() or s.dtype is not _U8 or s.shape != (t, k // 32) or not s.is_contiguous():
        raise ValueError("xq and xs: contiguous CUDA tensors, xs uint8 [t, k / 32] expected")
    return number, t, k


def _weights(q, s, k):
    """Rows of MXFP4 weights of k columns."""
    if q.dtype is not _U8 or q.dim() != 2 or q.shape[1] * 2 != k or not q.is_contiguous() or s.dtype is not _U8 or \
            s.shape != (q.shape[0], k // 32) or not s.is_contiguous():
        raise ValueError("weights: contiguous uint8 [n, k / 2] and [n, k / 32] of the activations' k expected")
    return q.shape[0]


def quantize_mx(x, format="e4m3", swiglu=False, out=None, stream=None):
    """(codes, scales) of bf16 rows [t, k], or with swiglu of SiLU(gate) * up
    of rows [t, 2 k] (gate first). Rows may be strided. out: (codes, scales) to write."""
    number = _format(format)
    if x.dtype is not _BF16 or x.dim() != 2 or not x.is_cuda or _strides(x)[1] not in (1, None):
        raise ValueError("x: bf16 CUDA tensor [t, k] with dense rows expected")
    t, width = x.shape
    _need(not swiglu or width % 2 == 0, "x: [t, 2 k] expected with swiglu")
    k = width // 2 if swiglu else width
    stride = x.stride(0) if t > 1 else width
    _need(stride >= width, "x: rows of their own expected, not an expanded tensor")
    device = x.get_device()
    q, s = _outputs(out, number, t, k, x.device, stream)
    _on_device(device, q, s)
    raw = _raw(stream, device, *(out or ()))
    rc = (step._L or _lib()).mxfp4_quantize_mx(x.data_ptr(), stride, t, k, bool(swiglu), number, q.data_ptr(), s.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_quantize_mx")
    return q, s


def residual_norm_mx(x, residual, weight, post_weight=None, post_bias=None, gate=None, bias=None, scale=1.0, eps=1e-6,
                     weight_offset=0.0, kind="rms", format="e4m3", out=None, residual_out=None, stream=None):
    """(codes, scales, r): residual_norm with y as MX codes. out: (codes, scales) to write."""
    number = _format(format)
    device = x.get_device()
    t, n, gate_stride = step._norm_arguments(x, residual, weight, post_weight, post_bias, gate, bias, residual_out, kind)
    q, s = _outputs(out, number, t, n, x.device, stream)
    _on_device(device, residual, weight, post_weight, post_bias, gate, bias, q, s, residual_out)
    r = _made(stream, (t, n), _BF16, x.device) if residual_out is None else residual_out
    raw = _raw(stream, device, *(out or ()), residual_out)
    rc = (step._L or _lib()).mxfp4_residual_norm_mx(
        x.data_ptr(), residual.data_ptr(), t, n, _ptr(post_weight), _ptr(post_bias), _ptr(gate), gate_stride, scale,
        weight.data_ptr(), _ptr(bias), weight_offset, eps, kind == "layer", number, q.data_ptr(), s.data_ptr(),
        r.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_residual_norm_mx")
    return q, s, r


def linear_mx(xq, xs, wq, ws, out=None, stream=None):
    """bf16 [t, n]: MX activations (codes, scales) times MXFP4 weights wq
    [n, k / 2], ws [n, k / 32], for any t. k a multiple of 128."""
    number, t, k = _codes(xq, xs)
    n = _weights(wq, ws, k)
    device = xq.get_device()
    _on_device(device, xs, wq, ws, out)
    if out is None:
        y = _made(stream, (t, n), _BF16, xq.device)
    else:
        _need(out.dtype is _BF16 and out.shape == (t, n) and out.is_contiguous(), "out: contiguous bf16 [t, n] expected")
        y = out
    raw = _raw(stream, device, out)
    rc = (step._L or _lib()).mxfp4_linear_mx(xq.data_ptr(), xs.data_ptr(), number, t, k, wq.data_ptr(), ws.data_ptr(), n,
                                        y.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_linear_mx")
    return y


def swiglu_mx(xq, xs, w1q, w1s, format="e4m3", out=None, stream=None):
    """(codes, scales) of SiLU(W1_gate x) * (W1_up x), [t, inter]: MX
    activations in, MX codes of `format` out; w1q [2 inter, k / 2] and w1s
    [2 inter, k / 32], gate rows first. out: (codes, scales) to write."""
    to = _format(format)
    number, t, k = _codes(xq, xs)
    rows = _weights(w1q, w1s, k)
    _need(rows % 64 == 0, "weights: [2 inter, ...] with inter a multiple of 32 expected")
    device = xq.get_device()
    q, s = _outputs(out, to, t, rows // 2, xq.device, stream)
    _on_device(device, xs, w1q, w1s, q, s)
    raw = _raw(stream, device, *(out or ()))
    rc = (step._L or _lib()).mxfp4_swiglu_mx(xq.data_ptr(), xs.data_ptr(), number, t, k, w1q.data_ptr(), w1s.data_ptr(),
                                        rows // 2, to, q.data_ptr(), s.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_swiglu_mx")
    return q, s
