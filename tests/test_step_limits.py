"""Sizes at the limits of what the step's entry points accept: refused before
any launch (no GPU needed), with the stand-in pointers never read."""
import ctypes

import pytest

import mxfp4_weight_streaming_gb300 as mx
from mxfp4_weight_streaming_gb300.step import KVBatchStruct, KVCacheStruct

P = 0x1000


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mxfp4_weight_streaming_gb300 import build
    build.build()
    return mx.load()


def attention(tokens, heads, kv_heads, ws=P):
    cache = KVCacheStruct(k=P, v=P, num_pages=8, layers=1, kv_heads=kv_heads, page_size=16, head_dim=64)
    batch = KVBatchStruct(q_start=P, seq_lens=P, block_table=P, table_width=4, batch=2, tokens=tokens, max_q=3, max_seq=60)
    return mx.load().mxfp4_attention(P, heads * 64, heads, ctypes.byref(cache), ctypes.byref(batch), 0.1, 0.0, 0, None, P,
                                     None, ws, 1 << 40, None)


def test_rows_of_a_kv_head_stay_below_31_bits():
    """2^24 tokens of 128 heads a group are 2^31 rows."""
    assert attention(1 << 24, 256, 2) == mx.MXFP4_ERR_SHAPE
    assert attention((1 << 24) - 1, 256, 2) == mx.MXFP4_ERR_SHAPE  # no room for a row tile's rounding up
    assert attention((1 << 24) - 2, 256, 2, ws=None) == mx.MXFP4_ERR_WORKSPACE  # the next check
    assert attention(1 << 24, 254, 2, ws=None) == mx.MXFP4_ERR_WORKSPACE


def test_positions_need_a_tree():
    cache = KVCacheStruct(k=P, v=P, num_pages=8, layers=1, kv_heads=2, page_size=16, head_dim=64)
    batch = KVBatchStruct(q_start=P, seq_lens=P, block_table=P, table_width=4, batch=2, tokens=4, max_q=3, max_seq=60)

    def at(tree, positions, ws=P):
        return mx.load().mxfp4_attention_at(P, 512, 8, ctypes.byref(cache), ctypes.byref(batch), 0.1, 0.0, 8, tree, positions,
                                            P, None, ws, 1 << 40, None)

    assert at(None, P) == mx.MXFP4_ERR_INVALID_ARG
    assert at(P, P + 2) == mx.MXFP4_ERR_ALIGN
    assert at(P, P, ws=None) == at(P, None, ws=None) == at(None, None, ws=None) == mx.MXFP4_ERR_WORKSPACE
