"""Many tokens at once (prompt chunks, large batches) over the C ABI:
activations as microscaled (MX) codes, and their products with MXFP4 weights
(include/mxfp4.h has the definitions). Argument marshalling only, as in the
rest of the binding.

MX codes of [t, k] activations are a pair of tensors: float8_e4m3fn [t, k] or
uint8 [t, k / 2] (E2M1, two a byte), and uint8 scales [t, k / 32]. All tensors
of a call lie on the current GPU. With stream= a call runs on that stream, and
the results it makes are that stream's memory.

linear_mx and swiglu_mx take weights from whatever ran before. linear, moe and
ffn read theirs ahead: E2M1 codes of residual_norm_mx or swiglu_mx have to be
waited for before they serve those as weights, quantize_mx's need not be.
"""
from __future__ import annotations

import ctypes

import torch

from . import step
from .step import _BF16, _E4M3, _elsewhere, _empty, _fail, _made, _norm_arguments, _on_device, _ptr, _stream_of

_U8 = torch.uint8
_FORMATS = {"e4m3": 0, "e2m1": 1}


# As in step.py, what every call does on the host is kept short: a small call
# is bound by it. Memory that a call makes itself needs no checks.
def _format(name):
    number = _FORMATS.get(name)
    if number is None:
        raise ValueError("format: 'e4m3' or 'e2m1' expected")
    return number


def _lib():
    return step._L or step._lib()


def _given(out, number, t, k, device):
    """The caller's (codes, scales) for t rows of k values, if they fit."""
    q, s = out
    dtype, width = (_E4M3, k) if number == 0 else (_U8, k // 2)
    if q.dtype is not dtype or q.shape != (t, width) or not q.is_contiguous() or s.dtype is not _U8 or \
            s.shape != (t, k // 32) or not s.is_contiguous():
        raise ValueError("out: contiguous codes (float8_e4m3fn [t, k] or uint8 [t, k / 2]) and uint8 scales [t, k / 32] expected")
    _on_device(device, q, s)
    return q, s


def _outputs(out, number, t, k, device, x, stream):
    """(codes, scales) for t rows of k values: the caller's, or new ones."""
    if out is not None:
        return _given(out, number, t, k, device)
    at = x.device
    if stream is None:
        return (_empty((t, k), dtype=_E4M3, device=at) if number == 0 else _empty((t, k // 2), dtype=_U8, device=at)), \
            _empty((t, k // 32), dtype=_U8, device=at)
    return _made(stream, (t, k) if number == 0 else (t, k // 2), _U8 if number else _E4M3, at), _made(stream, (t, k // 32), _U8, at)


def _operands(q, s, wq, ws):
    """(format, t, k, rows of the weights, device) of a product's operands."""
    dtype = q.dtype
    if dtype is not _E4M3 and dtype is not _U8 or q.dim() != 2 or wq.dim() != 2:
        raise ValueError("xq: float8_e4m3fn [t, k] or uint8 [t, k / 2], weights: uint8 [n, k / 2] expected")
    number = 0 if dtype is _E4M3 else 1
    t, width = q.shape
    n, half = wq.shape
    k = 2 * half
    if width != (half if number else k):
        raise ValueError("weights: [n, k / 2] of the activations' k expected")
    blocks = k // 32
    if s.dtype is not _U8 or ws.dtype is not _U8 or wq.dtype is not _U8 or s.shape != (t, blocks) or ws.shape != (n, blocks):
        raise ValueError("weights: uint8 [n, k / 2], scales: uint8 [t, k / 32] and [n, k / 32] expected")
    if not (q.is_contiguous() and s.is_contiguous() and wq.is_contiguous() and ws.is_contiguous()):
        raise ValueError("activations and weights: contiguous tensors expected")
    device = q.get_device()
    if device < 0 or device != step._current_device() or s.get_device() != device or wq.get_device() != device or \
            ws.get_device() != device:
        _elsewhere()
    return number, t, k, n, device


def quantize_mx(x, format="e4m3", swiglu=False, out=None, stream=None):
    """(codes, scales) of bf16 rows [t, k], or with swiglu of SiLU(gate) * up
    of rows [t, 2 k] (gate first). Rows may be strided. out: (codes, scales) to write."""
    number = _format(format)
    if x.dtype is not _BF16 or x.dim() != 2 or not x.is_cuda:
        raise ValueError("x: bf16 CUDA tensor [t, k] expected")
    t, width = x.shape
    stride, one = x.stride()
    if one != 1 and width > 1 or t > 1 and stride < width:
        raise ValueError("x: dense rows of their own expected")
    k = width
    if swiglu:
        if width & 1:
            raise ValueError("x: [t, 2 k] expected with swiglu")
        k = width // 2
    device = x.get_device()
    _on_device(device)
    q, s = _outputs(out, number, t, k, device, x, stream)
    raw = step._raw_stream(device) if stream is None else _stream_of(stream, *(out or ()))
    rc = _lib().mxfp4_quantize_mx(x.data_ptr(), stride if t > 1 else width, t, k, 1 if swiglu else 0, number,
                                  q.data_ptr(), s.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_quantize_mx")
    return q, s


def residual_norm_mx(x, residual, weight, post_weight=None, post_bias=None, gate=None, bias=None, scale=1.0, eps=1e-6,
                     weight_offset=0.0, kind="rms", format="e4m3", out=None, residual_out=None, stream=None):
    """(codes, scales, r): residual_norm with y as MX codes. out: (codes, scales) to write."""
    number = _format(format)
    t, n, gate_stride = _norm_arguments(x, residual, weight, post_weight, post_bias, gate, bias, residual_out, kind)
    device = x.get_device()
    _on_device(device, residual, weight, post_weight, post_bias, gate, bias, residual_out)
    q, s = _outputs(out, number, t, n, device, x, stream)
    r = _made(stream, x.shape, _BF16, x.device) if residual_out is None else residual_out
    raw = step._raw_stream(device) if stream is None else _stream_of(stream, residual_out, *(out or ()))
    rc = _lib().mxfp4_residual_norm_mx(
        x.data_ptr(), residual.data_ptr(), t, n, _ptr(post_weight), _ptr(post_bias), _ptr(gate), gate_stride, scale,
        weight.data_ptr(), _ptr(bias), weight_offset, eps, kind == "layer", number, q.data_ptr(), s.data_ptr(),
        r.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_residual_norm_mx")
    return q, s, r


def linear_mx(xq, xs, wq, ws, out=None, stream=None):
    """bf16 [t, n]: MX activations (codes, scales) times MXFP4 weights wq
    [n, k / 2], ws [n, k / 32], for any t. k a multiple of 128."""
    number, t, k, n, device = _operands(xq, xs, wq, ws)
    if out is None:
        y = _made(stream, (t, n), _BF16, xq.device)
    else:
        if out.dtype is not _BF16 or out.shape != (t, n) or not out.is_contiguous():
            raise ValueError("out: contiguous bf16 [t, n] expected")
        _on_device(device, out)
        y = out
    raw = step._raw_stream(device) if stream is None else _stream_of(stream, out)
    rc = _lib().mxfp4_linear_mx(xq.data_ptr(), xs.data_ptr(), number, t, k, wq.data_ptr(), ws.data_ptr(), n, y.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_linear_mx")
    return y


class MxPlan(ctypes.Structure):
    """mxfp4_mx_plan_t: how linear_mx and swiglu_mx cut a product."""
    _fields_ = [(name, ctypes.c_int32) for name in ("pair", "width", "split", "ctas", "ring_slots", "stage_bytes",
                                                     "token_rows", "scale_slots", "scale_bytes", "inbox_bytes", "smem_bytes")]


def linear_mx_plan(t, k, n, format="e4m3", swiglu=False, aligned_rows=True, max_smem=232448, clusters=None):
    """The plan for these sizes (swiglu: of swiglu_mx, n = inter) as a dict.
    clusters: how many clusters of 1 .. 8 CTAs are resident at once (9 numbers,
    the first unused; None: GB300's). Host only; raises Mxfp4Error when no plan fits."""
    plan = MxPlan()
    room = None if clusters is None else (ctypes.c_int32 * 9)(*clusters)
    rc = _lib().mxfp4_linear_mx_plan(t, k, n, _format(format), bool(swiglu), bool(aligned_rows), max_smem, room,
                                     ctypes.addressof(plan))
    if rc:
        _fail(rc, "mxfp4_linear_mx_plan")
    return {name: getattr(plan, name) for name, _ in MxPlan._fields_}


def swiglu_mx(xq, xs, w1q, w1s, format="e4m3", out=None, stream=None):
    """(codes, scales) of SiLU(W1_gate x) * (W1_up x), [t, inter]: MX
    activations in, MX codes of `format` out; w1q [2 inter, k / 2] and w1s
    [2 inter, k / 32], gate rows first. out: (codes, scales) to write."""
    to = _format(format)
    number, t, k, rows, device = _operands(xq, xs, w1q, w1s)
    if rows % 64:
        raise ValueError("weights: [2 inter, ...] with inter a multiple of 32 expected")
    q, s = _outputs(out, to, t, rows // 2, device, xq, stream)
    raw = step._raw_stream(device) if stream is None else _stream_of(stream, *(out or ()))
    rc = _lib().mxfp4_swiglu_mx(xq.data_ptr(), xs.data_ptr(), number, t, k, w1q.data_ptr(), w1s.data_ptr(), rows // 2, to,
                                q.data_ptr(), s.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_swiglu_mx")
    return q, s
