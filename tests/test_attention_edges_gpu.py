"""mxfp4_attention where calls go to their limits."""
import pytest
import torch

from gpu_cases import lib
from step_cases import E4M3, Paged
from test_attention_gpu import run

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


# -------------------------------------------------- many short items per CTA
@pytest.mark.parametrize("dim,kv,group,new,requests", [
    (64, 8, 8, 5, 160),   # 40 rows: one row tile, shared by both streams of products
    (128, 8, 8, 5, 160),
    (64, 8, 8, 20, 80),   # 160 rows: a row tile per stream
    (128, 8, 8, 20, 80),
    (128, 4, 16, 20, 160),  # 320 rows: two items a request and KV head
])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_many_short_items_in_a_row(dim, kv, group, new, requests, dtype):
    """Four and more items of one key tile in a row on every CTA, some of two or three between them; the same bits
    each time."""
    mx = lib()
    lens = [new + (i * 37) % (128 - new) if i % 9 else 130 + (i * 11) % 200 for i in range(requests)]
    pg = Paged(dim + new, lens, kv, dim, 32, dtype)
    out, q, cache, batch = run(pg, [new] * requests, kv * group, what=f"{requests} short requests")
    ws = mx.attention_workspace(kv * group, cache, batch)
    for _ in range(20):
        again = mx.attention(q, cache, batch, workspace=ws)
        assert mx.last_device_status() == mx.MXFP4_OK
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
