"""mxfp4_attention against its definition in float64: head layouts, lengths
from nothing to many tiles, page sizes, masks that leave rows empty, and NaN
or nonsense in every place that a query does not see."""
import math

import pytest
import torch

from gpu_cases import Guarded, lib
from step_cases import E4M3, Paged, attention_bound, attention_ref, check, gen, ints, randn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def run(pg, news, heads, seed=0, scale=None, softcap=0.0, window=0, tree=None, strided=False, what=""):
    mx = lib()
    t = sum(news)
    g = gen(seed + 1)
    wide = randn(g, t, heads * pg.dim + (2 * pg.kv_heads * pg.dim if strided else 0))
    q = wide[:, :heads * pg.dim].unflatten(1, (heads, pg.dim))
    cache, batch = pg.cache(mx), pg.batch(mx, news)
    out, lse = Guarded((t, heads, pg.dim), BF16), Guarded((t, heads), torch.float32)
    out.t.fill_(math.nan)
    lse.t.fill_(math.nan)
    need = mx.load().mxfp4_attention_workspace_size(heads, cache.ref, batch.ref)
    ws = Guarded((need,), torch.uint8)
    ws.t.fill_(0xFF)
    mx.attention(q, cache, batch, scale=scale, softcap=softcap, window=window, tree_mask=tree, out=out.t, lse=lse.t,
                 workspace=ws.t)
    for buf, name in ((out, "out"), (lse, "lse"), (ws, "workspace")):
        buf.check(f"{what}: {name}")
    assert mx.last_device_status() == mx.MXFP4_OK
    ref, lse_ref, mag = attention_ref(pg, q, pg.dim ** -0.5 if scale is None else scale, softcap, window, tree)
    check(out.t, ref, attention_bound(ref, mag, pg.dtype), what)
    none = torch.isneginf(lse_ref)
    assert torch.equal(torch.isneginf(lse.t), none), f"{what}: empty rows"
    # Scores are fp32 sums of up to 128 products: 1e-4 is far above their error.
    assert torch.all((lse.t.double() - lse_ref)[~none].abs() < 1e-4), f"{what}: lse"
    return out.t, q, cache, batch


HEADS = [(8, 1, 128), (7, 1, 128), (14, 2, 64), (4, 4, 128), (56, 8, 128), (16, 1, 64), (20, 1, 128), (40, 2, 64)]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("heads,kv,dim", HEADS)
def test_decode_head_layouts(heads, kv, dim, dtype):
    """One new token per request; lengths of one, around a tile and many tiles."""
    lens = [1, 15, 64, 65, 700]
    pg = Paged(heads + dim, lens, kv, dim, 32, dtype)
    run(pg, [1] * len(lens), heads, what=f"decode {heads}/{kv}x{dim} {dtype}")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(page, dtype):
    lens = [page - 1, page, page + 1, 5 * page + 3]
    pg = Paged(page, lens, 2, 128, page, dtype, interleave=True, junk=2 ** 31 - 1)
    run(pg, [3, 1, 4, 2], 6, strided=True, what=f"page {page}")


@pytest.mark.parametrize("news,lens", [
    ([4, 4, 4], [4, 5, 300]),          # the whole sequence is new; a token before it
    ([1, 0, 9, 2], [200, 77, 9, 130]),  # a request without new tokens
    ([33], [1000]), ([64, 1], [64, 2000]),
    ([130, 17], [130, 400]), ([257], [1500]),
    ([300, 1, 40], [300, 513, 1030]),
])
@pytest.mark.parametrize("heads,kv,dim,dtype", [(7, 1, 128, BF16), (8, 2, 64, E4M3), (8, 2, 64, BF16),
                                                (12, 4, 128, E4M3)])
def test_chunks(news, lens, heads, kv, dim, dtype):
    pg = Paged(sum(news) + heads, lens, kv, dim, 16, dtype)
    run(pg, news, heads, strided=True, what=f"chunk {news} of {lens}")


@pytest.mark.parametrize("window", [1, 16, 63, 64, 100, 1000])
@pytest.mark.parametrize("news,lens", [([1, 1], [40, 900]), ([5, 90], [333, 700]), ([200], [1100])])
def test_window(window, news, lens):
    """Tokens that every query's window has left may lie in pages given away: their table entries are -1 here."""
    pg = Paged(window, lens, 2, 128, 16)
    for b, (n, seq) in enumerate(zip(news, lens)):
        gone = max(0, seq - n - window + 1) // 16
        pg.table[b, :gone] = -1
    run(pg, news, 8, window=window, what=f"window {window} {news} of {lens}")


@pytest.mark.parametrize("cap", [1.0, 30.0])
@pytest.mark.parametrize("news", [[1, 3], [40, 150]])
def test_softcap(cap, news):
    pg = Paged(3, [300, 450], 1, 64, 32)
    run(pg, news, 6, softcap=cap, scale=0.7, what=f"cap {cap}")


@pytest.mark.parametrize("heads,kv,dim,dtype", [(7, 1, 128, BF16), (4, 2, 64, E4M3), (2, 2, 128, E4M3)])
@pytest.mark.parametrize("window", [0, 10])
def test_tree_masks(heads, kv, dim, dtype, window):
    """Random draft trees, a token that does not see itself, and words of 0: with nothing before the chunk those
    rows are empty."""
    news, lens = [8, 64, 3, 5, 1], [500, 64, 3, 17, 90]
    pg = Paged(window + dim, lens, kv, dim, 16, dtype)
    g = torch.Generator().manual_seed(window)
    words = []
    for n in news:
        m = []
        for j in range(n):
            parent = int(torch.randint(0, j, (1,), generator=g)) if j else None
            m.append((m[parent] if j else 0) | 1 << j)
        words += m
    words[9] = 0  # sees nothing: its request has no earlier tokens
    words[72] = 0
    words[73] = 1 << 2
    signed = [w - (1 << 64) if w >> 63 else w for w in words]
    tree = torch.tensor(signed, dtype=torch.int64, device="cuda")
    run(pg, news, heads, window=window, tree=tree, what=f"tree {dtype}")


def test_more_new_tokens_than_the_cache_holds():
    """A length below the chunk's: the first queries lie before the sequence and see nothing."""
    pg = Paged(5, [6, 0, 40], 1, 64, 16)
    run(pg, [10, 3, 2], 4, what="short sequence")


def test_many_requests_and_long_sequences():
    lens = [(i * 97) % 260 + 1 for i in range(300)]
    run(Paged(8, lens, 1, 64, 16), [1] * 300, 4, what="300 requests")
    run(Paged(9, [20011, 3], 2, 128, 64), [2, 1], 8, what="long")
    run(Paged(10, [9973], 1, 128, 64, E4M3), [4], 8, what="long e4m3")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("news,heads", [([6], 4), ([70], 8), ([200], 2)])
def test_not_finite_beyond_what_a_query_sees(dtype, news, heads):
    """The last new token's K and V are NaN: only its own row may notice."""
    mx = lib()
    n, seq = news[0], news[0] + 37
    pg = Paged(n, [seq], 2, 64, 16, dtype)
    p, r = int(pg.table[0, (seq - 1) // 16]), (seq - 1) % 16
    for pool in (pg.kp, pg.vp):
        if dtype == E4M3:
            pool.view(torch.uint8)[p, :, r] = 0x7F
        else:
            pool[p, :, r, ::2] = math.nan
            pool[p, :, r, 1::2] = math.inf
    q = randn(gen(2), n, heads, 64)
    out = mx.attention(q, pg.cache(mx), pg.batch(mx, news))
    ref, _, mag = attention_ref(pg, q[:, :], 0.125)
    check(out[:-1], ref[:-1], attention_bound(ref, mag, dtype)[:-1], "rows before the NaN token")
    assert torch.isnan(out[-1].float()).any()


def test_scores_far_from_zero_and_one_sided():
    """Scores of +-1e4 and a maximum that moves in every tile."""
    mx = lib()
    pg = Paged(4, [1000], 1, 64, 16)
    q = randn(gen(1), 3, 2, 64) * 0 + 1
    q[1] *= 40
    q[2] *= -40
    ramp = torch.arange(1000, device="cuda", dtype=torch.float32)[:, None, None] * 0.01
    k = (pg.k[0].float() * 0.1 + ramp).to(BF16)
    j = torch.arange(1000, device="cuda")
    pg.kp[pg.table[0].long()[j // 16], :, j % 16] = k
    pg.k[0] = k.double()
    batch = pg.batch(mx, [3])
    out = mx.attention(q, pg.cache(mx), batch, scale=1.0)
    ref, _, mag = attention_ref(pg, q, 1.0)
    # Scores up to 25600 are fp32 sums: off by up to 2^-23 of it, 0.003, which
    # moves a probability by as much of itself.
    check(out, ref, attention_bound(ref, mag) + 0.012 * mag, "large scores")


def test_repeats_bit_for_bit_and_on_another_stream():
    mx = lib()
    pg = Paged(6, [3000, 77, 512], 2, 128, 32)
    out, q, cache, batch = run(pg, [4, 1, 9], 14, what="first")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = mx.attention(q, cache, batch, stream=s)
    s.synchronize()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_lengths_change_under_a_captured_graph():
    mx = lib()
    pg = Paged(7, [900, 640], 2, 128, 64)
    pg.news, pg.start = [2, 3], [0, 2, 5]
    lens = ints([100, 64])
    batch = mx.KVBatch(ints([0, 2, 5]), lens, pg.table, tokens=5, max_q=3, max_seq=960)
    cache, q = pg.cache(mx), randn(gen(3), 5, 6, 128)
    ws, out = mx.attention_workspace(6, cache, batch), torch.empty(5, 6, 128, dtype=BF16, device="cuda")
    mx.attention(q, cache, batch, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.attention(q, cache, batch, out=out, workspace=ws)
    k, v = pg.k, pg.v
    for now in ([900, 3], [2, 640], [513, 512]):
        lens.copy_(ints(now))
        graph.replay()
        torch.cuda.synchronize()
        pg.lens, pg.k, pg.v = now, [x[:n] for x, n in zip(k, now)], [x[:n] for x, n in zip(v, now)]
        ref, _, mag = attention_ref(pg, q, 128 ** -0.5)
        check(out, ref, attention_bound(ref, mag), f"lengths {now}")


def test_pages_beyond_32_bit_offsets():
    """A pool of more than 2^32 elements, the tokens in its last pages."""
    mx = lib()
    page, kv, dim = 64, 8, 128
    pages = (1 << 32) // (page * kv * dim) + 9
    kp = torch.empty(pages, kv, page, dim, dtype=BF16, device="cuda")
    vp = torch.empty(pages, kv, page, dim, dtype=BF16, device="cuda")
    pg = Paged(11, [150], kv, dim, page, spare=0)
    order = torch.arange(pages - 3, pages, device="cuda")
    kp[order], vp[order] = pg.kp[pg.table[0].long()], pg.vp[pg.table[0].long()]
    pg.kp, pg.vp, pg.table = kp, vp, order.to(torch.int32)[None].contiguous()
    run(pg, [2], 16, what="far pages")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("news,heads,cap", [([8], 8, 0.0), ([200], 8, 30.0)])
def test_a_wait_that_runs_out_is_reported(dtype, news, heads, cap):
    """On a test-only build whose first K tile never arrives (and a limit of
    1 ms): the call ends, the status says so, and the product library's next
    call is right."""
    import ctypes

    from mxfp4_weight_streaming_gb300 import build
    mx = lib()
    path = build.build_test_variant("withhold", ["MXFP4_TEST_WITHHOLD_STAGE", "MXFP4_WAIT_LIMIT_NS=1000000ull"])
    other = ctypes.CDLL(path)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    other.mxfp4_attention.argtypes = [P, ctypes.c_int64, I, P, P, F, F, I, P, P, P, P, ctypes.c_size_t, P]
    other.mxfp4_last_device_status.argtypes = [P]
    pg = Paged(3, [news[0] + 700], 1, 128, 32, dtype)
    q = randn(gen(1), news[0], heads, 128)
    cache, batch = pg.cache(mx), pg.batch(mx, news)
    ws, out = mx.attention_workspace(heads, cache, batch), torch.empty_like(q)
    stream = torch.cuda.current_stream().cuda_stream
    rc = other.mxfp4_attention(q.data_ptr(), q.stride(0), heads, cache.ref, batch.ref, 0.1, cap, 0, None, out.data_ptr(),
                               None, ws.data_ptr(), ws.numel(), stream)
    assert rc == mx.MXFP4_OK
    assert other.mxfp4_last_device_status(stream) == mx.MXFP4_ERR_TIMEOUT
    assert other.mxfp4_last_device_status(stream) == mx.MXFP4_OK
    out = mx.attention(q, cache, batch, scale=0.1, softcap=cap, workspace=ws)
    assert mx.last_device_status() == mx.MXFP4_OK
    ref, _, mag = attention_ref(pg, q, 0.1, cap)
    check(out, ref, attention_bound(ref, mag, dtype), "after the timeout")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("page,dim", [(16, 128), (32, 64), (64, 128), (128, 64), (256, 128), (1024, 64)])
def test_page_sizes_with_many_rows(page, dim, dtype):
    """Pages smaller and larger than the 128-key tiles, K and V interleaved in one pool, nonsense in unused entries."""
    lens = [2 * page + 45, 47, page - 1 if page > 64 else 5 * page]
    pg = Paged(page + dim, lens, 2, dim, page, dtype, interleave=True, junk=-7)
    run(pg, [45, 47, 9], 8, strided=True, what=f"many rows, page {page}")
    run(pg, [45, 47, 9], 30, what=f"two row tiles, page {page}")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("news,heads", [([3, 1], 4), ([30, 2], 4), ([150, 7], 4)])
def test_negative_and_zero_scale(news, heads, dtype):
    for scale, cap in ((-0.1, 0.0), (-0.2, 5.0), (0.0, 0.0)):
        pg = Paged(news[0], [400, 77], 2, 64, 16, dtype)
        run(pg, news, heads, scale=scale, softcap=cap, what=f"scale {scale} cap {cap}")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_many_requests_with_many_rows(dtype):
    """More requests than the kernel counts one by one, of different lengths, some without new tokens."""
    news = [(i * 7) % 11 for i in range(130)]
    lens = [n + (i * 53) % 300 for i, n in enumerate(news)]
    run(Paged(21, lens, 1, 64, 16, dtype), news, 8, what="130 requests of up to 80 rows")


def test_far_pages_with_many_rows():
    page, kv, dim = 64, 8, 128
    pages = (1 << 32) // (page * kv * dim) + 9
    kp = torch.empty(pages, kv, page, dim, dtype=BF16, device="cuda")
    vp = torch.empty(pages, kv, page, dim, dtype=BF16, device="cuda")
    pg = Paged(12, [190], kv, dim, page, spare=0)
    order = torch.arange(pages - 3, pages, device="cuda")
    kp[order], vp[order] = pg.kp[pg.table[0].long()], pg.vp[pg.table[0].long()]
    pg.kp, pg.vp, pg.table = kp, vp, order.to(torch.int32)[None].contiguous()
    run(pg, [40], 16, what="far pages, many rows")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("heads", [97, 128])
def test_widest_groups(heads, dtype):
    pg = Paged(heads, [300, 20], 1, 64, 16, dtype)
    run(pg, [2, 5], heads, what=f"group of {heads}")
