"""The attention side of a decode / verify step over the C ABI: norms around
a block, rotary positions with the cache write, attention over the paged KV
cache, and the cache's pages between steps (include/mxfp4.h has the
definitions). Argument marshalling only, as in the rest of the binding.

`KVCache` and `KVBatch` hold tensors and the C structs that point into them;
a program makes them once and passes them to every call. Their tensors are
read on the device by each call, so their contents (lengths, page numbers)
may change between calls, their addresses may not. All tensors of a call lie
on the current GPU. With stream= a call runs on that stream, and the results
it makes are that stream's memory.
"""
from __future__ import annotations

import ctypes
import math

import torch

KV_BF16, KV_E4M3 = 0, 1

_BF16, _E4M3, _F32, _I32, _I64 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32, torch.int64
_empty = torch.empty
_MOST = 2 ** 31 - 1  # ctypes takes a larger number by its low bits
_L = None  # the loaded library, from the first call on


class KVCacheStruct(ctypes.Structure):
    """mxfp4_kv_cache_t"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
        [(n, ctypes.c_int64) for n in ("page_stride", "layer_stride", "num_pages")] + \
        [(n, ctypes.c_int32) for n in ("layers", "kv_heads", "page_size", "head_dim", "dtype", "reserved")]


class KVBatchStruct(ctypes.Structure):
    """mxfp4_kv_batch_t"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_start", "seq_lens", "block_table")] + \
        [("table_stride", ctypes.c_int64)] + \
        [(n, ctypes.c_int32) for n in ("table_width", "batch", "tokens", "max_q", "max_seq", "reserved")]


# A small call spends more time on the host than on the GPU, so what every
# call does here is kept short: the library is looked up once, checks are
# plain attribute reads, and the current stream is read as a raw handle (0.1
# us; torch.cuda.current_stream() makes an object in 2.9 us).
def _lib():
    global _L
    if _L is None:
        from . import load
        _L = load()
    return _L


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere():
    raise ValueError("every tensor of a call has to be on one GPU, the current one; one is on the host or on another GPU")


def _on_device(device, *tensors):
    """Each of these (or None) on `device`, which has to be the current GPU: the library's launch goes there."""
    if device != _current_device():
        _elsewhere()
    for t in tensors:
        if t is not None and t.get_device() != device:
            _elsewhere()


def _fail(rc: int, what: str):
    from . import Mxfp4Error
    raise Mxfp4Error(rc, what)


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ints(t, count, name, device):
    """An int32 vector or matrix the C side can take as it lies in memory."""
    if t.dtype is not _I32 or t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous int32 CUDA tensor of {count} expected, got {t.dtype} {list(t.shape)}")
    if t.get_device() != device:
        _elsewhere()


def _strides(t):
    """A tensor's strides, None where there is one entry only and its stride says nothing."""
    return [stride if size > 1 else None for size, stride in zip(t.shape, t.stride())]


def _row_stride(table):
    """Entries between a block table's rows. A row that several requests
    share by expand() has a stride of 0, which the C side takes as dense."""
    rows, width = table.shape
    if rows < 2:
        return width
    stride = table.stride(0)
    if stride < width:
        raise ValueError("block_table: rows of their own expected, not an expanded tensor")
    return stride


def _stream_object(stream):
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))


def _made(stream, shape, dtype, device):
    """Memory for a call's result, of the stream that will write it: memory of
    the current one may be what that stream's earlier work still uses."""
    if stream is None:
        return _empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream)):
        return _empty(shape, dtype=dtype, device=device)


def _stream_of(stream, *given):
    """The raw handle of a stream given by the caller. Tensors given to be
    written (or None) are kept until that stream's work on them is done."""
    stream = _stream_object(stream)
    for t in given:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


class KVCache:
    """K and V page pools [num_pages, kv_heads, page_size, head_dim], or of
    several layers [layers, num_pages, ...] (bf16 or float8_e4m3fn; pages and
    layers may be strided, e.g. K and V interleaved in one pool), with fp32
    scales [kv_heads] for an E4M3 cache. rope_append and attention work on
    one layer: `cache.layer(i)`."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _need(k.dim() in (4, 5) and k.shape == v.shape and k.dtype == v.dtype and _strides(k) == _strides(v),
              "k and v: pools of one shape, type and strides expected")
        _need(k.is_cuda and v.is_cuda and k.dtype in (torch.bfloat16, torch.float8_e4m3fn),
              "k and v: bf16 or float8_e4m3fn CUDA tensors expected")
        pages, heads, page, dim = k.shape[-4:]
        strides = _strides(k)
        _need(all(have in (want, None) for have, want in zip(strides[-3:], (page * dim, dim, 1))), "a page has to be dense")
        # A stride of 0 (an expanded tensor) would mean "dense" to the C side.
        _need(all(have is None or have >= heads * page * dim for have in strides[:-3]), "pages and layers may not share memory")
        e4m3 = k.dtype == torch.float8_e4m3fn
        for sc in (k_scale, v_scale):
            _need(sc is None or (e4m3 and sc.is_cuda and sc.dtype == torch.float32 and sc.shape == (heads,)
                                 and sc.is_contiguous()), "scales: float32 [kv_heads] of an E4M3 cache expected")
        self.device = k.get_device()
        for t in (v, k_scale, v_scale):
            _need(t is None or t.get_device() == self.device, "pools and scales: tensors of one GPU expected")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.layers = k.shape[0] if k.dim() == 5 else 1
        self.struct = KVCacheStruct(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), strides[-4] or heads * page * dim,
                                    (strides[0] or 0) if k.dim() == 5 else 0, pages, self.layers, heads, page, dim,
                                    KV_E4M3 if e4m3 else KV_BF16, 0)
        self.ref = ctypes.addressof(self.struct)

    def layer(self, i: int, k_scale=None, v_scale=None) -> "KVCache":
        """One layer of the pools, with that layer's scales (by default the cache's own)."""
        _need(self.k.dim() == 5, "a cache of several layers expected")
        return KVCache(self.k[i], self.v[i], self.k_scale if k_scale is None else k_scale,
                       self.v_scale if v_scale is None else v_scale)


class KVBatch:
    """A step's new tokens: q_start int32 [batch + 1], seq_lens int32 [batch]
    (new tokens included), block_table int32 [batch, width]; on the host the
    rows of the token arrays and bounds of a request's new tokens and length."""

    def __init__(self, q_start, seq_lens, block_table, tokens, max_q, max_seq):
        b = seq_lens.numel()
        self.device = device = block_table.get_device()
        _ints(seq_lens, b, "seq_lens", device)
        _ints(q_start, b + 1, "q_start", device)
        _need(block_table.is_cuda and block_table.dtype == torch.int32 and block_table.dim() == 2
              and block_table.shape[0] == b and _strides(block_table)[1] in (1, None),
              "block_table: int32 CUDA tensor [batch, width] expected")
        self.q_start, self.seq_lens, self.block_table = q_start, seq_lens, block_table
        self.batch, self.tokens, self.max_q, self.max_seq = b, int(tokens), min(int(max_q), _MOST), min(int(max_seq), _MOST)
        width = block_table.shape[1]
        stride = _row_stride(block_table)
        self.struct = KVBatchStruct(_ptr(q_start), _ptr(seq_lens), _ptr(block_table), stride, width, b, self.tokens,
                                    self.max_q, self.max_seq, 0)
        self.ref = ctypes.addressof(self.struct)


def residual_norm(x, residual, weight, post_weight=None, post_bias=None, gate=None, bias=None, scale=1.0, eps=1e-6,
                  weight_offset=0.0, kind="rms", out=None, residual_out=None, stream=None):
    """(y, r) of bf16 [tokens, n] x and residual: r = residual + scale * gate * u
    with u = x or norm(x) * post_weight + post_bias, and y = norm(r) * weight + bias.
    gate: [n] or [tokens, n]; kind "rms" or "layer"; weights count as weight + weight_offset."""
    shape = x.shape
    if len(shape) != 2 or x.dtype is not _BF16 or residual.dtype is not _BF16 or residual.shape != shape or \
            not x.is_cuda or not x.is_contiguous() or not residual.is_contiguous():
        raise ValueError("x and residual: contiguous bf16 CUDA tensors [tokens, n] expected")
    t, n = shape
    for w in (weight, post_weight, post_bias, bias):
        if w is not None and (w.dtype is not _BF16 or w.numel() != n or not w.is_contiguous()):
            raise ValueError("weights: contiguous bf16 [n] expected")
    gate_stride = 0
    if gate is not None:
        _need(gate.dtype is _BF16 and gate.shape in ((n,), (t, n)) and (gate.stride(-1) == 1 or n == 1),
              "gate: bf16 [n] or [tokens, n] expected")
        if gate.dim() == 2:
            gate_stride = gate.stride(0) if t > 1 else n
    for o in (out, residual_out):
        if o is not None and (o.dtype is not _BF16 or o.shape != shape or not o.is_contiguous()):
            raise ValueError("outputs: contiguous bf16 [tokens, n] expected")
    if kind != "rms" and kind != "layer":
        raise ValueError("kind: 'rms' or 'layer' expected")
    device = x.get_device()
    _on_device(device, residual, weight, post_weight, post_bias, gate, bias, out, residual_out)
    y = _made(stream, shape, _BF16, x.device) if out is None else out
    r = _made(stream, shape, _BF16, x.device) if residual_out is None else residual_out
    raw = _raw_stream(device) if stream is None else _stream_of(stream, out, residual_out)
    rc = (_L or _lib()).mxfp4_residual_norm(
        x.data_ptr(), residual.data_ptr(), t, n, None if post_weight is None else post_weight.data_ptr(),
        _ptr(post_bias), _ptr(gate), gate_stride, scale, weight.data_ptr(), _ptr(bias), weight_offset, eps,
        kind == "layer", y.data_ptr(), r.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_residual_norm")
    return y, r


def rope_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, trained=0, fast=32.0, slow=1.0,
                     device="cuda"):
    """(inv_freq float32 [rotary_dim / 2], factor) for rope_append.

    scaling None: base ** (-2j / rotary_dim). To stretch a model beyond the
    `trained` positions by `factor`:
      "linear"  every frequency divided by factor;
      "base"    the base raised so that the lowest frequency is divided by
                factor and the highest stays;
      "ramp"    frequencies that turn more than `fast` times over the trained
                positions stay, those that turn less than `slow` times are
                divided by factor, a linear ramp (over the pair's index)
                between, whose slow end may lie past the last pair (up to
                index rotary_dim - 1); q and k are scaled by 0.1 ln(factor) + 1
                (Peng et al., 2023).
    """
    _need(rotary_dim >= 2 and rotary_dim % 2 == 0 and factor > 0, "rotary_dim: even, factor: positive expected")
    _need(scaling in (None, "linear", "base", "ramp"), "scaling: None, 'linear', 'base' or 'ramp' expected")
    half = rotary_dim // 2
    if scaling == "base" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = [base ** (-2.0 * j / rotary_dim) for j in range(half)]
    amplitude = 1.0
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "ramp":
        _need(trained > 0 and fast > slow > 0, "trained positions and fast > slow > 0 expected")

        def pair_of(turns):  # the (fractional) pair that turns so often over the trained positions
            return rotary_dim * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), rotary_dim - 1)
        for j in range(half):
            stretched = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            freq[j] *= 1.0 - stretched + stretched / factor
        amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return torch.tensor(freq, dtype=torch.float64).float().to(device), amplitude


def rope_append(qkv, q_heads, inv_freq, cache, batch, interleaved=False, positions=None, factor=1.0, out=None,
                stream=None):
    """Turns q and k of the rows of qkv (bf16 [tokens, (q_heads + 2 kv_heads) *
    head_dim], q then k then v) by their positions, writes k and v to the
    cache and returns q, bf16 [tokens, q_heads, head_dim] (rows of no request
    are left as they are, uninitialised without out=). inv_freq float32
    [rotary_dim / 2] (None: only the cache write)."""
    tokens, d = batch.tokens, cache.head_dim
    if qkv.dtype is not _BF16 or qkv.shape != (tokens, (q_heads + 2 * cache.kv_heads) * d) or not qkv.is_cuda or \
            qkv.stride(1) != 1:
        raise ValueError("qkv: bf16 CUDA tensor [tokens, (q_heads + 2 kv_heads) * head_dim] expected")
    device = qkv.get_device()
    if cache.device != device or batch.device != device:
        _elsewhere()
    rotary = 0
    if inv_freq is not None:
        if inv_freq.dtype is not _F32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq: float32 CUDA tensor [rotary_dim / 2] expected")
        rotary = 2 * inv_freq.numel()
    if positions is not None:
        _ints(positions, tokens, "positions", device)
    _on_device(device, inv_freq, out)
    if out is None:
        q = _made(stream, (tokens, q_heads, d), _BF16, qkv.device)
    else:
        _need(out.dtype is _BF16 and out.shape == (tokens, q_heads, d) and out.is_contiguous(),
              "out: contiguous bf16 [tokens, q_heads, head_dim] expected")
        q = out
    raw = _raw_stream(device) if stream is None else _stream_of(stream, out)
    rc = (_L or _lib()).mxfp4_rope_append(
        qkv.data_ptr(), qkv.stride(0) if tokens > 1 else qkv.shape[1], q_heads, _ptr(positions), _ptr(inv_freq), rotary, interleaved, factor,
        cache.ref, batch.ref, q.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_rope_append")
    return q


def attention_workspace(q_heads, cache, batch):
    """Scratch for attention calls with this cache and batch (any lengths)."""
    return _attention_workspace(None, q_heads, cache, batch)


def _attention_workspace(stream, q_heads, cache, batch):
    nbytes = _lib().mxfp4_attention_workspace_size(q_heads, cache.ref, batch.ref)
    return _made(stream, max(nbytes, 256), torch.uint8, cache.k.device)


def attention(q, cache, batch, scale=None, softcap=0.0, window=0, tree_mask=None, out=None, lse=None, workspace=None,
              stream=None, positions=None):
    """bf16 [tokens, q_heads, head_dim]: attention of q (same shape, rows may
    be strided) over the cache; rows of no request are left as they are. scale defaults to head_dim ** -0.5; tree_mask
    int64 [tokens] (bit j: sees new token j); lse: float32 [tokens, q_heads] output.
    A window counts cache indices, or with a tree_mask the drafts' positions
    (int32 [tokens], as rope_append takes them)."""
    tokens, heads, d = shape = q.shape
    if q.dtype is not _BF16 or tokens != batch.tokens or d != cache.head_dim or not q.is_cuda:
        raise ValueError("q: bf16 CUDA tensor [tokens, q_heads, head_dim] expected")
    stride, head_stride, one = q.stride()
    _need(one == 1 and (head_stride == d or heads == 1), "q: dense rows expected")
    if tree_mask is not None:
        _need(tree_mask.dtype is _I64 and tree_mask.shape == (tokens,) and tree_mask.is_contiguous(),
              "tree_mask: int64 [tokens] expected")
    device = q.get_device()
    if cache.device != device or batch.device != device:
        _elsewhere()
    if positions is not None:
        _need(tree_mask is not None, "positions: a tree_mask expected too")
        _ints(positions, tokens, "positions", device)
    _on_device(device, tree_mask, out, lse, workspace)
    if out is None:
        o = _made(stream, shape, _BF16, q.device)
    else:
        _need(out.dtype is _BF16 and out.shape == shape and out.is_contiguous(),
              "out: contiguous bf16 [tokens, q_heads, head_dim] expected")
        o = out
    if lse is not None:
        _need(lse.dtype is _F32 and lse.shape == shape[:2] and lse.is_contiguous(),
              "lse: contiguous float32 [tokens, q_heads] expected")
    ws = _attention_workspace(stream, heads, cache, batch) if workspace is None else workspace
    if window > _MOST:
        window = _MOST
    raw = _raw_stream(device) if stream is None else _stream_of(stream, out, lse, workspace)
    if positions is None:
        rc = (_L or _lib()).mxfp4_attention(
            q.data_ptr(), stride if tokens > 1 else heads * d, heads, cache.ref, batch.ref,
            d ** -0.5 if scale is None else scale, softcap, window, _ptr(tree_mask), o.data_ptr(), _ptr(lse),
            ws.data_ptr(), ws.nbytes, raw)
    else:
        rc = (_L or _lib()).mxfp4_attention_at(
            q.data_ptr(), stride if tokens > 1 else heads * d, heads, cache.ref, batch.ref,
            d ** -0.5 if scale is None else scale, softcap, window, _ptr(tree_mask), positions.data_ptr(),
            o.data_ptr(), _ptr(lse), ws.data_ptr(), ws.nbytes, raw)
    if rc:
        _fail(rc, "mxfp4_attention")
    return o


def cache_workspace(sequences, num_pages, device="cuda"):
    """Scratch for cache_update calls of up to these sizes."""
    return _cache_workspace(None, sequences, num_pages, device)


def _cache_workspace(stream, sequences, num_pages, device):
    return _made(stream, _lib().mxfp4_cache_workspace_size(sequences, num_pages), torch.uint8, device)


def cache_update(cache, block_table, seq_lens, parent, keep, grow, workspace=None, stream=None):
    """The cache's pages for the next step: new sequence i continues
    parent[i] (negative: begins empty), cut to keep[i] tokens (keep None:
    all), with room for grow[i] more. Returns (block_table, seq_lens, copies,
    info): int32 [n, width], [n], [n, 3] for cache_copy, and [pages left
    free, pages asked for in vain]. A step captured in a CUDA graph copies
    table and lengths to the tensors of its KVBatch."""
    n, old, device = parent.numel(), seq_lens.numel(), block_table.get_device()
    _ints(parent, n, "parent", device)
    _ints(grow, n, "grow", device)
    _ints(seq_lens, old, "seq_lens", device)
    if keep is not None:
        _ints(keep, n, "keep", device)
    if block_table.dtype is not _I32 or block_table.dim() != 2 or block_table.shape[0] != old or \
            (block_table.stride(1) != 1 and block_table.shape[1] > 1) or not block_table.is_cuda:
        raise ValueError("block_table: int32 CUDA tensor [old, width] expected")
    _on_device(device, workspace)
    width, stride = block_table.shape[1], _row_stride(block_table)
    # Four allocations take 6 us of host time, one that is split and viewed 12.
    dev = block_table.device
    table = _made(stream, (n, width), _I32, dev)
    lens = _made(stream, n, _I32, dev)
    copies = _made(stream, (n, 3), _I32, dev)
    info = _made(stream, 2, _I32, dev)
    ws = _cache_workspace(stream, n, cache.num_pages, dev) if workspace is None else workspace
    raw = _raw_stream(device) if stream is None else _stream_of(stream, workspace)
    rc = (_L or _lib()).mxfp4_cache_update(
        block_table.data_ptr(), stride, width, seq_lens.data_ptr(), old,
        parent.data_ptr(), _ptr(keep), grow.data_ptr(), n, cache.num_pages, cache.page_size, table.data_ptr(),
        lens.data_ptr(), copies.data_ptr(), info.data_ptr(), ws.data_ptr(), ws.nbytes, raw)
    if rc:
        _fail(rc, "mxfp4_cache_update")
    return table, lens, copies, info


def cache_copy(cache, copies, stream=None):
    """Copies the page rows that cache_update lists, in every layer of the cache."""
    n, device = copies.shape[0], cache.device
    _ints(copies, 3 * n, "copies", device)
    _on_device(device)
    raw = _raw_stream(device) if stream is None else _stream_of(stream)
    rc = (_L or _lib()).mxfp4_cache_copy(cache.ref, copies.data_ptr(), n, raw)
    if rc:
        _fail(rc, "mxfp4_cache_copy")


def cache_accept(cache, batch, path, n_accept, out=None, stream=None):
    """Moves the rows of the accepted path (int32 [batch, path_len], indices
    among a request's new tokens; n_accept int32 [batch]) to the front of its
    new tokens, in every layer. Returns the lengths with the accepted tokens, int32 [batch]."""
    n, length, device = batch.batch, path.shape[1], cache.device
    _ints(path, n * length, "path", device)
    _ints(n_accept, n, "n_accept", device)
    if batch.device != device:
        _elsewhere()
    _on_device(device)
    if out is None:
        lens = _made(stream, n, _I32, path.device)
    else:
        _ints(out, n, "out", device)
        lens = out
    raw = _raw_stream(device) if stream is None else _stream_of(stream, out)
    rc = (_L or _lib()).mxfp4_cache_accept(cache.ref, batch.ref, path.data_ptr(), length, n_accept.data_ptr(),
                                           lens.data_ptr(), raw)
    if rc:
        _fail(rc, "mxfp4_cache_accept")
    return lens
