"""What the Python binding of the step's attention side refuses, and what it
passes on, seen without a GPU: tensors that say they are on one, and a stand-in
for the library that records the calls."""
import pytest
import torch

import mxfp4_weight_streaming_gb300 as mx
from mxfp4_weight_streaming_gb300 import step

BF16, I32 = torch.bfloat16, torch.int32


class OnGpu:
    """A tensor of host memory that says it is on GPU `device` (-1: on the host)."""

    def __init__(self, t, device=0):
        self.t, self.device_index = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    is_cuda = property(lambda self: self.device_index >= 0)

    def get_device(self):
        return self.device_index


class Library:
    """Takes the place of libmxfp4.so: every call succeeds and is recorded."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 256 if name.endswith("workspace_size") else 0
        return call


@pytest.fixture(autouse=True)
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(step, "_L", lib)
    monkeypatch.setattr(step, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(step, "_current_device", lambda: 0, raising=False)
    return lib


def ints(*shape, device=0):
    return OnGpu(torch.zeros(shape, dtype=I32), device)


def pools(layers=None, pages=8, heads=2, page=16, dim=64, device=0):
    shape = (() if layers is None else (layers,)) + (pages, heads, page, dim)
    return [OnGpu(torch.zeros(shape, dtype=BF16), device) for _ in range(2)]


# ------------------------------------------------------------------- strides
def test_expanded_tables_are_refused():
    """One row for every request has a stride of 0, which the C side takes as rows next to one another."""
    row = torch.zeros(1, 4, dtype=I32)
    with pytest.raises(ValueError):
        mx.KVBatch(ints(4), ints(3), OnGpu(row.expand(3, 4)), tokens=3, max_q=1, max_seq=60)
    batch = mx.KVBatch(ints(2), ints(1), OnGpu(row.expand(1, 4)), tokens=3, max_q=1, max_seq=60)  # a single row
    assert batch.struct.table_stride == 4
    wide = OnGpu(torch.zeros(3, 9, dtype=I32)[:, :4])
    assert mx.KVBatch(ints(4), ints(3), wide, tokens=3, max_q=1, max_seq=60).struct.table_stride == 9


def test_expanded_tables_are_refused_by_cache_update(library):
    cache = mx.KVCache(*pools())
    row = torch.zeros(1, 4, dtype=I32)
    ws = OnGpu(torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mx.cache_update(cache, OnGpu(row.expand(3, 4)), ints(3), ints(2), None, ints(2), workspace=ws)
    assert not library.calls


@pytest.mark.parametrize("layers", [None, 3])
def test_expanded_pools_are_refused(layers):
    """Pages (or layers) that are all the same memory."""
    one = torch.zeros(1, 2, 16, 64, dtype=BF16)
    if layers is None:
        same = [OnGpu(one.expand(8, -1, -1, -1)) for _ in range(2)]
    else:
        same = [OnGpu(torch.zeros(1, 8, 2, 16, 64, dtype=BF16).expand(3, -1, -1, -1, -1)) for _ in range(2)]
    with pytest.raises(ValueError):
        mx.KVCache(*same)
    if layers is None:
        assert mx.KVCache(*[OnGpu(one) for _ in range(2)]).struct.page_stride == 2 * 16 * 64


# ------------------------------------------------------------------- devices
def bf16(*shape, device=0):
    return OnGpu(torch.zeros(shape, dtype=BF16), device)


def a_batch(device=0, width=4):
    return mx.KVBatch(ints(3, device=device), ints(2, device=device), ints(2, width, device=device), tokens=4, max_q=2,
                      max_seq=60)


def norm_call(**kw):
    a = dict(x=bf16(4, 64), residual=bf16(4, 64), weight=bf16(64), post_weight=bf16(64), post_bias=bf16(64),
             gate=bf16(4, 64), bias=bf16(64), out=bf16(4, 64), residual_out=bf16(4, 64))
    return mx.residual_norm, dict(a, **kw)


def rope_call(**kw):
    a = dict(qkv=bf16(4, 8 * 64), q_heads=4, inv_freq=OnGpu(torch.zeros(32)), cache=mx.KVCache(*pools()),
             batch=a_batch(), positions=ints(4), out=bf16(4, 4, 64))
    return mx.rope_append, dict(a, **kw)


def attention_call(**kw):
    a = dict(q=bf16(4, 4, 64), cache=mx.KVCache(*pools()), batch=a_batch(),
             tree_mask=OnGpu(torch.zeros(4, dtype=torch.int64)), out=bf16(4, 4, 64), lse=OnGpu(torch.zeros(4, 4)),
             workspace=OnGpu(torch.zeros(256, dtype=torch.uint8)))
    return mx.attention, dict(a, **kw)


def update_call(**kw):
    a = dict(cache=mx.KVCache(*pools()), block_table=ints(2, 4), seq_lens=ints(2), parent=ints(3), keep=ints(3),
             grow=ints(3), workspace=OnGpu(torch.zeros(256, dtype=torch.uint8)))
    return mx.cache_update, dict(a, **kw)


def copy_call(**kw):
    return mx.cache_copy, dict(dict(cache=mx.KVCache(*pools()), copies=ints(2, 3)), **kw)


def accept_call(**kw):
    a = dict(cache=mx.KVCache(*pools()), batch=a_batch(), path=ints(2, 3), n_accept=ints(2), out=ints(2))
    return mx.cache_accept, dict(a, **kw)


CALLS = dict(norm=norm_call, rope=rope_call, attention=attention_call, update=update_call, copy=copy_call,
             accept=accept_call)
OPERANDS = [(name, key) for name, make in CALLS.items() for key, v in make()[1].items()
            if isinstance(v, (OnGpu, mx.KVCache, mx.KVBatch))]


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_one_gpu_go_through(name, library):
    f, a = CALLS[name]()
    f(**a)
    assert len(library.calls) == 1


@pytest.mark.parametrize("name,key", [x for x in OPERANDS if x != ("update", "cache")])
@pytest.mark.parametrize("device", [-1, 1])
def test_an_operand_elsewhere_is_refused(name, key, device, library):
    """One tensor (or cache, or batch) on the host or on another GPU."""
    f, a = CALLS[name]()
    if key == "cache":
        if device < 0:
            return  # a cache on the host cannot be made
        a[key] = mx.KVCache(*pools(device=device))
    elif key == "batch":
        if device < 0:
            return
        a[key] = a_batch(device=device)
    else:
        a[key] = OnGpu(a[key].t, device)
    with pytest.raises(ValueError):
        f(**a)
    assert not library.calls


@pytest.mark.parametrize("name", CALLS)
def test_another_current_gpu_is_refused(name, library, monkeypatch):
    f, a = CALLS[name]()
    monkeypatch.setattr(step, "_current_device", lambda: 1)
    with pytest.raises(ValueError):
        f(**a)
    assert not library.calls


def test_handles_over_two_devices_are_refused():
    k, v = pools()
    with pytest.raises(ValueError):
        mx.KVCache(k, OnGpu(v.t, 1))
    e = [OnGpu(p.t.to(torch.float8_e4m3fn)) for p in (k, v)]
    with pytest.raises(ValueError):
        mx.KVCache(*e, k_scale=OnGpu(torch.ones(2), 1))
    for bad in range(3):
        args = [ints(3), ints(2), ints(2, 4)]
        args[bad] = OnGpu(args[bad].t, 1)
        with pytest.raises(ValueError):
            mx.KVBatch(*args, tokens=4, max_q=2, max_seq=60)


def test_the_row_stride_of_a_single_token_does_not_matter(library):
    batch = mx.KVBatch(ints(2), ints(1), ints(1, 4), tokens=1, max_q=1, max_seq=60)
    row = torch.zeros(8 * 64, dtype=BF16).as_strided((1, 8 * 64), (3, 1))
    f, a = rope_call(qkv=OnGpu(row), batch=batch, positions=None, out=bf16(1, 4, 64))
    f(**a)
    assert library.calls[-1][1][1] == 8 * 64
    q = torch.zeros(4 * 64, dtype=BF16).as_strided((1, 4, 64), (3, 64, 1))
    f, a = attention_call(q=OnGpu(q), batch=batch, tree_mask=None, out=bf16(1, 4, 64), lse=None)
    f(**a)
    assert library.calls[-1][1][1] == 4 * 64


def test_numbers_beyond_32_bits_are_cut_not_wrapped(library):
    f, a = attention_call(window=2 ** 32 + 5)
    f(**a)
    assert library.calls[-1][1][7] == 2 ** 31 - 1
    loose = mx.KVBatch(ints(3), ints(2), ints(2, 4), tokens=4, max_q=2 ** 32 + 1, max_seq=2 ** 40)
    assert (loose.struct.max_q, loose.struct.max_seq) == (2 ** 31 - 1, 2 ** 31 - 1)


# ------------------------------------------------------------------- streams
class Stream:
    cuda_stream = 77


@pytest.mark.parametrize("name", CALLS)
def test_results_are_memory_of_the_stream_that_writes_them(name, library, monkeypatch):
    """Memory of the current stream's pool may still be in use by that stream's earlier work, which another stream
    does not wait for."""
    import contextlib
    current, made, kept = [0], [], []

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream.cuda_stream
        yield
        current[0] = before

    def empty(*shape, dtype, device):
        made.append(current[0])
        return torch.zeros(*shape, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(step, "_empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda x: empty(x.shape, dtype=x.dtype, device=x.device))
    monkeypatch.setattr(OnGpu, "record_stream", lambda self, s: kept.append(s.cuda_stream), raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    f, a = CALLS[name]()
    f(**a, stream=Stream())  # what is given to be written is kept
    given = [k for k in ("out", "residual_out", "lse", "workspace") if k in a]
    assert kept == [77] * len(given) and library.calls[-1][1][-1] == 77
    made.clear()
    f(**{k: v for k, v in a.items() if k not in ("out", "residual_out", "workspace")}, stream=Stream())
    assert set(made) <= {77} and (made or name == "copy")


# -------------------------------------------------------- sizes of one
def test_strides_of_single_entries_do_not_matter():
    """A dimension of size 1 may carry any stride: out of a transpose, or of a slice of a larger pool."""
    k = torch.zeros(8, 16, 1, 64, dtype=BF16).transpose(1, 2)  # one KV head: stride(1) is a row's
    v = torch.zeros(8, 1, 16, 64, dtype=BF16)
    c = mx.KVCache(OnGpu(k), OnGpu(v)).struct
    assert k.stride() != v.stride() and (c.page_stride, c.kv_heads, c.layer_stride) == (16 * 64, 1, 0)
    one_page = torch.zeros(4, 2, 16, 64, dtype=BF16).as_strided((1, 2, 16, 64), (8, 1024, 64, 1))
    c = mx.KVCache(OnGpu(one_page), OnGpu(torch.zeros(1, 2, 16, 64, dtype=BF16))).struct
    assert c.num_pages == 1 and c.page_stride in (0, 2 * 16 * 64)
    one_layer = torch.zeros(1, 8, 2, 16, 64, dtype=BF16).as_strided((1, 8, 2, 16, 64), (4, 2048, 1024, 64, 1))
    c = mx.KVCache(*[OnGpu(one_layer)] * 2).struct
    assert c.layers == 1 and c.layer_stride in (0, 8 * 2048)
    with pytest.raises(ValueError):  # strides that matter still have to agree
        mx.KVCache(OnGpu(torch.zeros(8, 2, 2, 16, 64, dtype=BF16)[:, 0]), OnGpu(torch.zeros(8, 2, 16, 64, dtype=BF16)))
    with pytest.raises(ValueError):
        mx.KVCache(*[OnGpu(torch.zeros(8, 16, 2, 64, dtype=BF16).transpose(1, 2))] * 2)


def test_a_table_of_one_column_and_a_gate_of_one_element():
    table = torch.zeros(40, dtype=I32).as_strided((3, 1), (4, 7))
    assert mx.KVBatch(ints(4), ints(3), OnGpu(table), tokens=3, max_q=1, max_seq=16).struct.table_stride == 4
    f, a = norm_call(x=bf16(4, 1), residual=bf16(4, 1), weight=bf16(1), post_weight=None, post_bias=None, bias=None,
                     gate=OnGpu(torch.zeros(4, 8, dtype=BF16).as_strided((4, 1), (8, 3))), out=bf16(4, 1),
                     residual_out=bf16(4, 1))
    f(**a)


# ----------------------------------------------------------------- positions
def test_positions_of_drafts(library):
    f, a = attention_call(positions=ints(4))
    f(**a)
    assert library.calls[-1][0] == "mxfp4_attention_at"
    for bad in (dict(tree_mask=None), dict(positions=ints(5)), dict(positions=ints(4, device=-1))):
        library.calls.clear()
        f, a = attention_call(**dict(dict(positions=ints(4)), **bad))
        with pytest.raises(ValueError):
            f(**a)
        assert not library.calls


# ------------------------------------------------------------- rotary ramp
@pytest.mark.parametrize("dim,base,trained,factor", [(128, 1e4, 131072, 4.0), (128, 1e4, 4096, 8.0), (64, 1e4, 32768, 4.0),
                                                     (128, 5e5, 8192, 16.0), (32, 1e4, 10 ** 6, 2.0)])
def test_ramp_of_rope_frequencies(dim, base, trained, factor):
    """A pair's share of the stretch by the turns it makes over the trained
    positions, from the definition: none above 32, all below 1, linear in the
    pair's index between the pairs that turn so often (whole indices around
    them, the slow one at most rotary_dim - 1)."""
    import math
    freq, _ = mx.rope_frequencies(dim, base=base, scaling="ramp", factor=factor, trained=trained, device="cpu")

    def index(turns):
        return dim / 2 * math.log(trained / (turns * 2 * math.pi), base)

    lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), dim - 1)
    for j in range(dim // 2):
        plain = base ** (-2 * j / dim)
        share = min(max((j - lo) / (hi - lo), 0.0), 1.0)
        want = plain * ((1 - share) + share / factor)
        assert abs(freq[j].item() - want) <= 1e-6 * want, j
        if trained * plain / (2 * math.pi) > 32.0:
            assert abs(freq[j].item() - plain) <= 1e-6 * plain
        if trained * plain / (2 * math.pi) > 1.0:  # still turns: not stretched in full
            assert freq[j].item() > plain / factor * (1 + 1e-6)
