"""Argument checks of the step's attention-side entry points: every refusal
comes before any launch (these calls need no GPU), and the binding's structs
have the header's layout."""
import ctypes

import pytest

import mxfp4_weight_streaming_gb300 as mx
from mxfp4_weight_streaming_gb300.step import KVBatchStruct, KVCacheStruct

P, ODD = 0x1000, 0x1001  # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mxfp4_weight_streaming_gb300 import build
    build.build()
    return mx.load()


def cache(**kw):
    base = dict(k=P, v=P, page_stride=0, layer_stride=0, num_pages=8, layers=1, kv_heads=2, page_size=16,
                head_dim=64, dtype=0, reserved=0)
    return KVCacheStruct(**{**base, **kw})


def batch(**kw):
    base = dict(q_start=P, seq_lens=P, block_table=P, table_stride=0, table_width=4, batch=2, tokens=4, max_q=3,
                max_seq=60, reserved=0)
    return KVBatchStruct(**{**base, **kw})


def call(f, names, base, change):
    a = dict(base, **change)
    return getattr(mx.load(), f)(*[ctypes.byref(a[n]) if isinstance(a[n], ctypes.Structure) else a[n] for n in names])


BAD_CACHE = [(dict(k=None), 1), (dict(v=None), 1), (dict(num_pages=0), 1), (dict(layers=0), 1), (dict(kv_heads=0), 1),
             (dict(dtype=2), 1), (dict(reserved=1), 1), (dict(page_stride=-8), 1), (dict(page_size=24), 2),
             (dict(page_size=8), 2), (dict(page_size=2048), 2), (dict(head_dim=96), 2), (dict(num_pages=1 << 24), 2),
             (dict(layers=1025), 2), (dict(page_stride=2 * 16 * 64 - 8), 2), (dict(k=ODD), 3),
             (dict(page_stride=2 * 16 * 64 + 1), 3), (dict(k_scale=ODD), 3), (dict(layer_stride=(1 << 20) + 4), 3)]
BAD_BATCH = [(dict(q_start=None), 1), (dict(seq_lens=None), 1), (dict(block_table=None), 1), (dict(batch=0), 1),
             (dict(tokens=0), 1), (dict(table_width=0), 1), (dict(max_q=0), 1), (dict(max_seq=0), 1),
             (dict(reserved=2), 1), (dict(batch=1025), 2), (dict(table_stride=3), 2), (dict(seq_lens=ODD), 3)]

ATT = ["q", "q_stride", "heads", "cache", "batch", "scale", "softcap", "window", "tree", "out", "lse", "ws", "bytes", "stream"]
ATT_BASE = dict(q=P, q_stride=8 * 64, heads=8, scale=0.1, softcap=0.0, window=0, tree=None, out=P, lse=None, ws=P,
                bytes=1 << 40, stream=None)
ROPE = ["qkv", "stride", "heads", "pos", "freq", "rotary", "inter", "factor", "cache", "batch", "out", "stream"]
ROPE_BASE = dict(qkv=P, stride=12 * 64, heads=8, pos=None, freq=P, rotary=64, inter=0, factor=1.0, out=P, stream=None)


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_bad_caches(change, status):
    for f, names, base in (("mxfp4_attention", ATT, ATT_BASE), ("mxfp4_rope_append", ROPE, ROPE_BASE)):
        assert call(f, names, base, dict(cache=cache(**change), batch=batch())) == status, f
    assert call("mxfp4_cache_copy", ["c", "p", "n", "s"], dict(p=P, n=1, s=None), dict(c=cache(**change))) == status
    assert mx.load().mxfp4_cache_copy(None, P, 1, None) == 1


@pytest.mark.parametrize("change,status", BAD_BATCH)
def test_bad_batches(change, status):
    for f, names, base in (("mxfp4_attention", ATT, ATT_BASE), ("mxfp4_rope_append", ROPE, ROPE_BASE)):
        assert call(f, names, base, dict(cache=cache(), batch=batch(**change))) == status, f
    names = ["c", "b", "path", "len", "n", "out", "s"]
    base = dict(c=cache(), path=P, len=4, n=P, out=P + 64, s=None)
    assert call("mxfp4_cache_accept", names, base, dict(b=batch(**change))) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(heads=0), 1), (dict(window=-1), 1), (dict(softcap=-1.0), 1),
    (dict(softcap=float("nan")), 1), (dict(softcap=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(q_stride=8 * 64 - 8), 1), (dict(heads=7), 2), (dict(heads=258, q_stride=258 * 64), 2), (dict(q=ODD), 3),
    (dict(q_stride=8 * 64 + 4), 3), (dict(out=ODD), 3), (dict(lse=ODD), 3), (dict(tree=P + 4), 3), (dict(ws=None), 4),
    (dict(ws=P + 128), 3), (dict(bytes=100), 4)])
def test_attention_refusals(change, status):
    assert call("mxfp4_attention", ATT, ATT_BASE, dict(dict(cache=cache(), batch=batch()), **change)) == status


def test_attention_tree_of_more_than_64():
    assert call("mxfp4_attention", ATT, ATT_BASE, dict(cache=cache(), batch=batch(max_q=65), tree=P)) == 2
    assert mx.load().mxfp4_attention_workspace_size(7, ctypes.byref(cache()), ctypes.byref(batch())) == 0
    assert mx.load().mxfp4_attention_workspace_size(8, ctypes.byref(cache()), ctypes.byref(batch())) > 0


@pytest.mark.parametrize("change,status", [
    (dict(qkv=None), 1), (dict(out=None), 1), (dict(heads=0), 1), (dict(freq=None), 1), (dict(rotary=-2), 1),
    (dict(stride=12 * 64 - 8), 1), (dict(rotary=63), 2), (dict(rotary=66), 2), (dict(qkv=ODD), 3),
    (dict(stride=12 * 64 + 2), 3), (dict(pos=ODD), 3), (dict(out=P + 8), 3)])
def test_rope_refusals(change, status):
    assert call("mxfp4_rope_append", ROPE, ROPE_BASE, dict(dict(cache=cache(), batch=batch()), **change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(res=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(r=None), 1), (dict(t=0), 1),
    (dict(n=0), 1), (dict(pb=P, pw=None), 1), (dict(gs=32), 1), (dict(eps=-1.0), 1), (dict(y=P, r=P), 1),
    (dict(n=32769), 2), (dict(x=ODD), 3), (dict(gate=ODD), 3)])
def test_norm_refusals(change, status):
    names = ["x", "res", "t", "n", "pw", "pb", "gate", "gs", "scale", "w", "b", "off", "eps", "layer", "y", "r", "s"]
    base = dict(x=P, res=P, t=2, n=64, pw=P, pb=None, gate=None, gs=0, scale=1.0, w=P, b=None, off=0.0, eps=1e-6,
                layer=0, y=P, r=P + 4096, s=None)
    assert call("mxfp4_residual_norm", names, base, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(table=None), 1), (dict(lens=None), 1), (dict(parent=None), 1), (dict(grow=None), 1), (dict(out=None), 1),
    (dict(copies=None), 1), (dict(info=None), 1), (dict(width=0), 1), (dict(old=0), 1), (dict(n=0), 1),
    (dict(pages=0), 1), (dict(out=P), 1), (dict(lens_out=P), 1), (dict(n=65537), 2), (dict(page=48), 2),
    (dict(stride=3), 2), (dict(pages=1 << 24), 2), (dict(width=1 << 22, page=512), 2), (dict(parent=ODD), 3),
    (dict(ws=None), 4), (dict(ws=P + 16), 3), (dict(bytes=64), 4)])
def test_cache_update_refusals(change, status):
    names = ["table", "stride", "width", "lens", "old", "parent", "keep", "grow", "n", "pages", "page", "out",
             "lens_out", "copies", "info", "ws", "bytes", "s"]
    base = dict(table=P, stride=0, width=4, lens=P, old=2, parent=P, keep=None, grow=P, n=2, pages=8, page=16,
                out=P + 256, lens_out=P + 512, copies=P + 1024, info=P + 2048, ws=P, bytes=1 << 20, s=None)
    assert call("mxfp4_cache_update", names, base, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(path=None), 1), (dict(n=None), 1), (dict(out=None), 1), (dict(len=0), 1), (dict(out=P), 1),
    (dict(len=65), 2), (dict(path=ODD), 3)])
def test_cache_accept_refusals(change, status):
    names = ["c", "b", "path", "len", "n", "out", "s"]
    base = dict(c=cache(), b=batch(), path=P, len=4, n=P, out=P + 64, s=None)
    assert call("mxfp4_cache_accept", names, base, change) == status


def test_cache_copy_refusals():
    f = mx.load().mxfp4_cache_copy
    c = cache()
    assert f(ctypes.byref(c), None, 1, None) == 1 and f(ctypes.byref(c), P, 0, None) == 1
    assert f(ctypes.byref(c), P, 65537, None) == 2 and f(ctypes.byref(c), ODD, 1, None) == 3


def test_binding_refuses_wrong_tensors():
    import torch
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mx.residual_norm(x, x, x[0])
    with pytest.raises(ValueError):
        mx.KVCache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64))
    with pytest.raises(ValueError):
        mx.rope_frequencies(7)
    with pytest.raises(ValueError):
        mx.rope_frequencies(8, scaling="ramp")


def test_struct_layout():
    """Offsets a C compiler gives the header's structs."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [(KVCacheStruct, "mxfp4_kv_cache_t"), (KVBatchStruct, "mxfp4_kv_batch_t")]
    lines = [f'printf("%zu\\n", sizeof({c}));' + "".join(f'printf("%zu\\n", offsetof({c}, {n}));' for n, _ in s._fields_)
             for s, c in fields]
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "a.c")
        with open(src, "w") as f:
            f.write('#include <stdio.h>\n#include <stddef.h>\n#include "mxfp4.h"\nint main(void){' + "".join(lines) + "return 0;}")
        subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), src, "-o", os.path.join(d, "a")])
        got = [int(x) for x in subprocess.check_output([os.path.join(d, "a")]).split()]
    want = []
    for s, _ in fields:
        want += [ctypes.sizeof(s)] + [getattr(s, n).offset for n, _ in s._fields_]
    assert got == want
