"""mxfp4_attention where calls go to their limits."""
import math

import pytest
import torch

from gpu_cases import lib
from step_cases import E4M3, Paged, attention_bound, attention_ref, check, gen, ints, randn
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


# ----------------------------------------------------- NaN and capped scores
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("news,heads", [([1], 8), ([5], 8), ([30], 8), ([70], 8)])
def test_visible_nan_reaches_the_output(news, heads, cap, dtype):
    """A NaN in a key that every query sees makes the outputs of its KV head
    NaN, a NaN in q those of its own row; the rest stays right."""
    mx = lib()
    n, seq = news[0], news[0] + 90
    pg = Paged(n + 50, [seq], 2, 64, 16, dtype)
    q = randn(gen(n), n, heads, 64)
    cache, batch = pg.cache(mx), pg.batch(mx, news)
    ref, _, mag = attention_ref(pg, q, 0.125, cap)
    bound = attention_bound(ref, mag, dtype)

    bad = q.clone()
    bad[n - 1, heads - 1, 5] = math.nan
    out = mx.attention(bad, cache, batch, softcap=cap)
    assert torch.isnan(out[n - 1, heads - 1].float()).all()
    keep = torch.ones(n, heads, dtype=torch.bool, device="cuda")
    keep[n - 1, heads - 1] = False
    check(out[keep], ref[keep], bound[keep], "rows without the NaN")

    p, r = int(pg.table[0, 40 // 16]), 40 % 16  # key 40, KV head 0
    if dtype == E4M3:
        pg.kp.view(torch.uint8)[p, 0, r, 3] = 0x7F
    else:
        pg.kp[p, 0, r, 3] = math.nan
    out = mx.attention(q, cache, batch, softcap=cap)
    assert torch.isnan(out[:, :heads // 2].float()).all()
    check(out[:, heads // 2:], ref[:, heads // 2:], bound[:, heads // 2:], "the other KV head")


# ------------------------------------------------------------ a head's scale
@pytest.mark.parametrize("news,heads", [([3, 1], 4), ([30, 2], 4), ([150, 7], 4)])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("scale", [0.2, -0.2])
def test_negative_and_zero_scales_of_a_head(news, heads, cap, scale):
    """Element * scale of its KV head, whatever the scale's sign."""
    pg = Paged(news[0] + 7, [400, 77], 3, 64, 16, E4M3)
    for head, f in ((0, -1.0), (1, 0.0)):
        pg.k_scale[head] *= f
        pg.k = [k * torch.where(torch.arange(3, device="cuda") == head, f, 1.0)[:, None] for k in pg.k]
    pg.v_scale[2] *= -1
    pg.v = [v * torch.where(torch.arange(3, device="cuda") == 2, -1.0, 1.0)[:, None] for v in pg.v]
    run(pg, news, heads * 3, scale=scale, softcap=cap, what=f"scales of heads, cap {cap}")


@pytest.mark.parametrize("news", [[3], [40], [150]])
def test_nan_scale_of_a_head(news):
    """Its scores are NaN, and so is every row that sees a key; a row that sees none stays 0."""
    mx = lib()
    pg = Paged(5, [news[0] - 1], 2, 64, 16, E4M3)  # the first query lies before the sequence
    pg.k_scale[1] = math.nan
    q = randn(gen(3), news[0], 8, 64)
    out = mx.attention(q, pg.cache(mx), pg.batch(mx, news))
    pg.k_scale = pg.k_scale.nan_to_num(1.0)
    pg.k = [k.nan_to_num(0.0) for k in pg.k]
    ref, _, mag = attention_ref(pg, q, 0.125)
    check(out[:, :4], ref[:, :4], attention_bound(ref, mag, E4M3)[:, :4], "the other KV head")
    assert torch.isnan(out[1:, 4:].float()).all() and (out[0] == 0).all()


# ------------------------------------------------------------------- bounds
@pytest.mark.parametrize("window", [2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("heads", [1, 4, 16])
def test_windows_longer_than_any_sequence(window, dtype, heads):
    """Also where the first queries lie before their sequence."""
    pg = Paged(heads, [6, 0, 40], 1, 64, 16, dtype)
    run(pg, [10, 3, 2], heads, window=window, what=f"window {window}")


def test_bounds_far_above_the_lengths():
    """max_q and max_seq size the kernels; any int32 will do."""
    mx = lib()
    lens = [(i * 7) % 90 + 3 for i in range(1024)]
    pg = Paged(31, lens, 8, 64, 16)
    news = [i % 3 for i in range(1024)]
    tight = pg.batch(mx, news)
    start, most = ints(pg.start), 2 ** 31 - 1
    loose = mx.KVBatch(start, ints(lens), pg.table, tokens=pg.start[-1], max_q=most, max_seq=most)
    q = randn(gen(4), pg.start[-1], 64, 64)
    a, b = mx.attention(q, pg.cache(mx), tight), mx.attention(q, pg.cache(mx), loose)
    # Two kernels: each off by what attention_bound allows, 2^-7 + 2^-12 of the largest |v| (below 6) at most.
    assert (a.double() - b.double()).abs().max() < 2 * (2 ** -7 + 2 ** -12) * 6


# ------------------------------------------------- windows of a tree's drafts
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("window", [1, 5, 70, 130, 4000])
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 128), (2, 2, 64), (8, 1, 128), (16, 1, 64)])
def test_window_counts_from_a_drafts_position(heads, kv, dim, window, dtype):
    """A draft of depth d sees the keys before the step that decoding it after its ancestors alone would see; which
    new tokens it sees is the mask's, also where the window is shorter than the path."""
    mx = lib()
    news, lens = [16, 40, 3, 1, 7], [700, 171, 3, 90, 9]
    pg = Paged(window + heads, lens, kv, dim, 16, dtype)
    g = torch.Generator().manual_seed(window)
    words, depths = [], []
    for n in news:
        m, d = [], []
        for j in range(n):
            parent = int(torch.randint(max(0, j - 4), j, (1,), generator=g)) if j else None
            m.append((m[parent] if j else 0) | 1 << j)
            d.append(d[parent] + 1 if j else 0)
        words += m
        depths += d
    words[20] = 0
    t = sum(news)
    q = randn(gen(window), t, heads, dim)
    batch = pg.batch(mx, news)
    first = [seq - n for seq, n in zip(lens, news) for _ in range(n)]
    positions = ints([f + d for f, d in zip(first, depths)])
    tree = torch.tensor(words, dtype=torch.int64, device="cuda")
    out = mx.attention(q, pg.cache(mx), batch, window=window, tree_mask=tree, positions=positions)
    ref = torch.zeros(t, heads, dim, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for b, n in enumerate(news):
        for i in range(n):
            row, start = pg.start[b] + i, lens[b] - n
            see = torch.zeros(lens[b], dtype=torch.bool, device="cuda")
            see[max(0, start + depths[row] - window + 1):start] = True
            for j in range(n):
                see[start + j] = bool(words[row] >> j & 1)
            if not see.any():
                continue
            k, v = (x[b][see].repeat_interleave(heads // kv, 1) for x in (pg.k, pg.v))
            p = torch.softmax(torch.einsum("hd,jhd->hj", q[row].double(), k) * dim ** -0.5, 1)
            ref[row] = torch.einsum("hj,jhd->hd", p, v)
            mag[row] = torch.einsum("hj,jhd->hd", p, v.abs())
    check(out, ref, attention_bound(ref, mag, dtype), f"window {window}")
    # Positions beyond the request's new tokens count as the nearest of them.
    high = mx.attention(q, pg.cache(mx), batch, window=window, tree_mask=tree, positions=positions + 10 ** 6)
    last = ints([f + n - 1 for f, n in zip(first, (n for n in news for _ in range(n)))])
    same = mx.attention(q, pg.cache(mx), batch, window=window, tree_mask=tree, positions=last)
    assert torch.equal(high.view(torch.int16), same.view(torch.int16))
