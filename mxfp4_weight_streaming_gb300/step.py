"""The attention side of a decode / verify step over the C ABI: norms around
a block, rotary positions with the cache write, attention over the paged KV
cache, and the cache's pages between steps (include/mxfp4.h has the
definitions). Argument marshalling only, as in the rest of the binding.

`KVCache` and `KVBatch` hold tensors and the C structs that point into them;
a program makes them once and passes them to every call. Their tensors are
read on the device by each call, so their contents (lengths, page numbers)
may change between calls, their addresses may not.
"""
from __future__ import annotations

import ctypes
import math

KV_BF16, KV_E4M3 = 0, 1


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


def _lib():
    from . import load
    return load()


def _check(rc: int, what: str):
    if rc:
        from . import Mxfp4Error
        raise Mxfp4Error(rc, what)


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _int32(t, shape, name):
    import torch
    _need(t.is_cuda and t.dtype == torch.int32 and tuple(t.shape) == tuple(shape) and t.is_contiguous(),
          f"{name}: contiguous int32 CUDA tensor {list(shape)} expected, got {t.dtype} {list(t.shape)}")


def _stream_of(stream, *made):
    """The raw stream to launch on. Tensors made for the call are kept for a
    stream that is not torch's current one until its work is done."""
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    for t in made:
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
        import torch
        _need(k.dim() in (4, 5) and k.shape == v.shape and k.dtype == v.dtype and k.stride() == v.stride(),
              "k and v: pools of one shape, type and strides expected")
        _need(k.is_cuda and v.is_cuda and k.dtype in (torch.bfloat16, torch.float8_e4m3fn),
              "k and v: bf16 or float8_e4m3fn CUDA tensors expected")
        pages, heads, page, dim = k.shape[-4:]
        _need(k.stride(-1) == 1 and k.stride(-2) == dim and k.stride(-3) == page * dim, "a page has to be dense")
        e4m3 = k.dtype == torch.float8_e4m3fn
        for sc in (k_scale, v_scale):
            _need(sc is None or (e4m3 and sc.is_cuda and sc.dtype == torch.float32 and sc.shape == (heads,)
                                 and sc.is_contiguous()), "scales: float32 [kv_heads] of an E4M3 cache expected")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.layers = k.shape[0] if k.dim() == 5 else 1
        self.struct = KVCacheStruct(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), k.stride(-4),
                                    k.stride(0) if k.dim() == 5 else 0, pages, self.layers, heads, page, dim,
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
        import torch
        b = seq_lens.numel()
        _int32(seq_lens, (b,), "seq_lens")
        _int32(q_start, (b + 1,), "q_start")
        _need(block_table.is_cuda and block_table.dtype == torch.int32 and block_table.dim() == 2
              and block_table.shape[0] == b and block_table.stride(1) == 1,
              "block_table: int32 CUDA tensor [batch, width] expected")
        self.q_start, self.seq_lens, self.block_table = q_start, seq_lens, block_table
        self.batch, self.tokens, self.max_q, self.max_seq = b, int(tokens), int(max_q), int(max_seq)
        width = block_table.shape[1]
        stride = block_table.stride(0) if b > 1 else width
        self.struct = KVBatchStruct(_ptr(q_start), _ptr(seq_lens), _ptr(block_table), stride, width, b, self.tokens,
                                    self.max_q, self.max_seq, 0)
        self.ref = ctypes.addressof(self.struct)


def residual_norm(x, residual, weight, post_weight=None, post_bias=None, gate=None, bias=None, scale=1.0, eps=1e-6,
                  weight_offset=0.0, kind="rms", out=None, residual_out=None, stream=None):
    """(y, r) of bf16 [tokens, n] x and residual: r = residual + scale * gate * u
    with u = x or norm(x) * post_weight + post_bias, and y = norm(r) * weight + bias.
    gate: [n] or [tokens, n]; kind "rms" or "layer"; weights count as weight + weight_offset."""
    import torch
    _need(kind in ("rms", "layer"), "kind: 'rms' or 'layer' expected")
    bf = torch.bfloat16
    _need(x.dim() == 2 and x.is_cuda and x.dtype == bf and x.is_contiguous() and residual.shape == x.shape
          and residual.dtype == bf and residual.is_contiguous(), "x and residual: contiguous bf16 [tokens, n] expected")
    t, n = x.shape
    for w in (weight, post_weight, post_bias, bias):
        _need(w is None or (w.dtype == bf and w.shape == (n,) and w.is_contiguous()), "weights: bf16 [n] expected")
    gate_stride = 0
    if gate is not None:
        _need(gate.dtype == bf and gate.shape in ((n,), (t, n)) and gate.stride(-1) == 1,
              "gate: bf16 [n] or [tokens, n] expected")
        if gate.dim() == 2:
            gate_stride = gate.stride(0)
    for o in (out, residual_out):
        _need(o is None or (o.dtype == bf and o.shape == x.shape and o.is_contiguous()),
              "outputs: contiguous bf16 [tokens, n] expected")
    y = torch.empty_like(x) if out is None else out
    r = torch.empty_like(x) if residual_out is None else residual_out
    _check(_lib().mxfp4_residual_norm(x.data_ptr(), residual.data_ptr(), t, n, _ptr(post_weight), _ptr(post_bias),
                                      _ptr(gate), gate_stride, scale, weight.data_ptr(), _ptr(bias), weight_offset,
                                      eps, kind == "layer", y.data_ptr(), r.data_ptr(),
                                      _stream_of(stream, None if out is not None else y,
                                                 None if residual_out is not None else r)), "mxfp4_residual_norm")
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
                between; q and k are scaled by 0.1 ln(factor) + 1.
    """
    import torch
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

        lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), half - 1)
        for j in range(half):
            stretched = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            freq[j] *= 1.0 - stretched + stretched / factor
        amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return torch.tensor(freq, dtype=torch.float64).float().to(device), amplitude


def rope_append(qkv, q_heads, inv_freq, cache, batch, interleaved=False, positions=None, factor=1.0, out=None,
                stream=None):
    """Turns q and k of the rows of qkv (bf16 [tokens, (q_heads + 2 kv_heads) *
    head_dim], q then k then v) by their positions, writes k and v to the
    cache and returns q, bf16 [tokens, q_heads, head_dim]. inv_freq float32
    [rotary_dim / 2] (None: only the cache write)."""
    import torch
    d = cache.head_dim
    _need(qkv.is_cuda and qkv.dtype == torch.bfloat16 and qkv.dim() == 2 and qkv.stride(1) == 1
          and tuple(qkv.shape) == (batch.tokens, (q_heads + 2 * cache.kv_heads) * d),
          "qkv: bf16 [tokens, (q_heads + 2 kv_heads) * head_dim] expected")
    _need(inv_freq is None or (inv_freq.is_cuda and inv_freq.dtype == torch.float32 and inv_freq.is_contiguous()
                               and inv_freq.dim() == 1), "inv_freq: float32 [rotary_dim / 2] expected")
    if positions is not None:
        _int32(positions, (batch.tokens,), "positions")
    _need(out is None or (out.dtype == torch.bfloat16 and out.shape == (batch.tokens, q_heads, d)
                          and out.is_contiguous()), "out: contiguous bf16 [tokens, q_heads, head_dim] expected")
    q = torch.empty((batch.tokens, q_heads, d), dtype=torch.bfloat16, device=qkv.device) if out is None else out
    _check(_lib().mxfp4_rope_append(qkv.data_ptr(), qkv.stride(0), q_heads, _ptr(positions), _ptr(inv_freq),
                                    0 if inv_freq is None else 2 * inv_freq.numel(), interleaved, factor, cache.ref,
                                    batch.ref, q.data_ptr(), _stream_of(stream, None if out is not None else q)),
           "mxfp4_rope_append")
    return q


def attention_workspace(q_heads, cache, batch):
    """Scratch for attention calls with this cache and batch (any lengths)."""
    import torch
    nbytes = _lib().mxfp4_attention_workspace_size(q_heads, cache.ref, batch.ref)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=cache.k.device)


def attention(q, cache, batch, scale=None, softcap=0.0, window=0, tree_mask=None, out=None, lse=None, workspace=None,
              stream=None):
    """bf16 [tokens, q_heads, head_dim]: attention of q (same shape, rows may
    be strided) over the cache. scale defaults to head_dim ** -0.5; tree_mask
    int64 [tokens] (bit j: sees new token j); lse: float32 [tokens, q_heads] output."""
    import torch
    d = cache.head_dim
    _need(q.is_cuda and q.dtype == torch.bfloat16 and q.dim() == 3 and q.shape[0] == batch.tokens
          and q.shape[2] == d and q.stride(2) == 1 and q.stride(1) == d,
          "q: bf16 [tokens, q_heads, head_dim] with dense rows expected")
    heads = q.shape[1]
    _need(tree_mask is None or (tree_mask.dtype == torch.int64 and tree_mask.shape == (batch.tokens,)
                                and tree_mask.is_contiguous()), "tree_mask: int64 [tokens] expected")
    _need(out is None or (out.dtype == torch.bfloat16 and out.shape == q.shape and out.is_contiguous()),
          "out: contiguous bf16 [tokens, q_heads, head_dim] expected")
    _need(lse is None or (lse.dtype == torch.float32 and lse.shape == q.shape[:2] and lse.is_contiguous()),
          "lse: contiguous float32 [tokens, q_heads] expected")
    o = torch.empty((batch.tokens, heads, d), dtype=torch.bfloat16, device=q.device) if out is None else out
    ws = attention_workspace(heads, cache, batch) if workspace is None else workspace
    _check(_lib().mxfp4_attention(q.data_ptr(), q.stride(0) if batch.tokens > 1 else heads * d, heads, cache.ref,
                                  batch.ref, d ** -0.5 if scale is None else scale, softcap, window, _ptr(tree_mask),
                                  o.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(),
                                  _stream_of(stream, None if out is not None else o,
                                             None if workspace is not None else ws)), "mxfp4_attention")
    return o


def cache_workspace(sequences, num_pages, device="cuda"):
    """Scratch for cache_update calls of up to these sizes."""
    import torch
    return torch.empty(_lib().mxfp4_cache_workspace_size(sequences, num_pages), dtype=torch.uint8, device=device)


def cache_update(cache, block_table, seq_lens, parent, keep, grow, workspace=None, stream=None):
    """The cache's pages for the next step: new sequence i continues
    parent[i] (negative: begins empty), cut to keep[i] tokens (keep None:
    all), with room for grow[i] more. Returns (block_table, seq_lens, copies,
    info): int32 [n, width], [n], [n, 3] for cache_copy, and [pages left
    free, pages asked for in vain]."""
    import torch
    n, old = parent.numel(), seq_lens.numel()
    _int32(parent, (n,), "parent")
    _int32(grow, (n,), "grow")
    _int32(seq_lens, (old,), "seq_lens")
    if keep is not None:
        _int32(keep, (n,), "keep")
    _need(block_table.is_cuda and block_table.dtype == torch.int32 and block_table.dim() == 2
          and block_table.shape[0] == old and block_table.stride(1) == 1, "block_table: int32 [old, width] expected")
    width = block_table.shape[1]
    dev = block_table.device
    made = torch.empty(n * (width + 4) + 2, dtype=torch.int32, device=dev)  # one allocation for the four outputs
    table, lens, copies, info = made.split((n * width, n, 3 * n, 2))
    table, copies = table.view(n, width), copies.view(n, 3)
    ws = cache_workspace(n, cache.num_pages, dev) if workspace is None else workspace
    _check(_lib().mxfp4_cache_update(block_table.data_ptr(), block_table.stride(0) if old > 1 else width, width,
                                     seq_lens.data_ptr(), old, parent.data_ptr(), _ptr(keep), grow.data_ptr(), n,
                                     cache.num_pages, cache.page_size, table.data_ptr(), lens.data_ptr(),
                                     copies.data_ptr(), info.data_ptr(), ws.data_ptr(), ws.numel(),
                                     _stream_of(stream, made, None if workspace is not None else ws)),
           "mxfp4_cache_update")
    return table, lens, copies, info


def cache_copy(cache, copies, stream=None):
    """Copies the page rows that cache_update lists, in every layer of the cache."""
    _int32(copies, (copies.shape[0], 3), "copies")
    _check(_lib().mxfp4_cache_copy(cache.ref, copies.data_ptr(), copies.shape[0], _stream_of(stream)),
           "mxfp4_cache_copy")


def cache_accept(cache, batch, path, n_accept, out=None, stream=None):
    """Moves the rows of the accepted path (int32 [batch, path_len], indices
    among a request's new tokens; n_accept int32 [batch]) to the front of its
    new tokens, in every layer. Returns the lengths with the accepted tokens, int32 [batch]."""
    import torch
    _int32(path, (batch.batch, path.shape[1]), "path")
    _int32(n_accept, (batch.batch,), "n_accept")
    if out is not None:
        _int32(out, (batch.batch,), "out")
    lens = torch.empty(batch.batch, dtype=torch.int32, device=path.device) if out is None else out
    _check(_lib().mxfp4_cache_accept(cache.ref, batch.ref, path.data_ptr(), path.shape[1], n_accept.data_ptr(),
                                     lens.data_ptr(), _stream_of(stream, None if out is not None else lens)),
           "mxfp4_cache_accept")
    return lens
