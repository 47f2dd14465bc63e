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
