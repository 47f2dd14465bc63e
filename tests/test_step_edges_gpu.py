"""The step's norms, rotary positions and page bookkeeping where calls go to
their limits."""
import math

import pytest
import torch

from gpu_cases import lib
from step_cases import E4M3, Paged, check, gen, ints, randn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


# ------------------------------------------------------------------- streams
def test_results_on_another_stream_are_not_memory_of_the_current_ones_work():
    """The current stream still has to write into memory that the host has given back; a call on another stream,
    which does not wait for that, may not be handed it."""
    mx = lib()
    g = gen(1)
    x, res, w = randn(g, 64, 4096), randn(g, 64, 4096), randn(g, 4096)
    y0, r0 = mx.residual_norm(x, res, w)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    late = [torch.empty_like(x).fill_(7) for _ in range(2)]
    del late
    y, r = mx.residual_norm(x, res, w, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(r, r0)


# --------------------------------------------------------------------- pages
def test_more_pages_asked_for_than_32_bits_count():
    """130 sequences that ask for 2^24 - 1 pages each, 2^31 in all, of a pool of 9: the first takes them, the others
    get nothing, and none reads beyond the list of free pages."""
    mx = lib()
    n, width = 130, (1 << 24) - 1
    pool = torch.empty(9, 1, 16, 64, dtype=BF16, device="cuda")
    old = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    grow = 2 ** 31 - 1
    table, lens, copies, info = mx.cache_update(mx.KVCache(pool, pool), old, ints([0]), ints([-1] * n), None,
                                                ints([grow] * n))
    assert table[0, :9].tolist() == list(range(9)) and int((table[0, 9:] != -1).sum()) == 0
    assert all(int((row != -1).sum()) == 0 for row in table[1:])
    assert lens.tolist() == [9 * 16] + [0] * (n - 1) and copies.tolist() == [[-1, -1, 0]] * n
    assert info.tolist() == [0, 2 ** 31 - 1]
    small = mx.cache_update(mx.KVCache(pool, pool), old[:, :4].contiguous(), ints([0]), ints([-1] * 3), None, ints([40] * 3))
    assert small[3].tolist() == [0, 0] and small[1].tolist() == [40] * 3


# --------------------------------------------------------------------- norms
def test_residual_norm_of_as_many_rows_as_an_int_counts():
    """2^31 - 1 rows of one element: y = sign(r) but for eps, r = x + residual."""
    mx = lib()
    t = 2 ** 31 - 1
    x = torch.empty(t, 1, dtype=BF16, device="cuda")
    x.view(-1)[:-1].view(-1, 2).copy_(torch.tensor([1.0, -3.0], dtype=BF16, device="cuda"))
    x[-1] = 5.0
    w = torch.full((1,), 2.0, dtype=BF16, device="cuda")
    y, r = mx.residual_norm(x, x, w, out=torch.full_like(x, 9.0), residual_out=torch.full_like(x, 9.0))
    torch.cuda.synchronize()
    for got, even, odd, last in ((r, 2.0, -6.0, 10.0), (y, 2.0, -2.0, 2.0)):
        pairs = got.view(-1)[:-1].view(-1, 2)
        for part in pairs.split(1 << 27):
            assert bool((part[:, 0] == even).all()) and bool((part[:, 1] == odd).all())
        assert float(got[-1]) == last


# --------------------------------------------------------- accepted drafts
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_accept_where_the_sequence_is_shorter_than_the_chunk(dtype):
    """New token i lies at seq_len - n + i here too: those below 0 are not in the cache, and move nothing."""
    mx = lib()
    lens, news = [6, 0, 20], [10, 3, 4]
    pg = Paged(2, lens, 2, 64, 16, dtype, layers=2)
    for pool in (pg.kp, pg.vp):
        b = pool.view(torch.uint8)
        b.copy_(torch.randint(0, 255, b.shape, dtype=torch.uint8, device="cuda", generator=gen(3)))
    path = torch.tensor([[0, 1, 2, 3, 9, 7, 5, 4], [0, 1, 2, 0, 0, 0, 0, 0], [0, 2, 3, 0, 0, 0, 0, 0]], dtype=torch.int32)
    took = [8, 3, 3]
    old = {n: getattr(pg, n).view(torch.uint8).clone() for n in ("kp", "vp")}
    out = mx.cache_accept(pg.cache(mx), pg.batch(mx, news), path.cuda(), ints(took))
    assert out.tolist() == [6 - 10 + 8, 0, 19]
    for name in ("kp", "vp"):
        want = old[name].clone()
        for b in range(3):
            first = lens[b] - news[b]
            for i in range(took[b]):
                to, fr = first + i, first + int(path[b, i])
                if to >= 0 and fr >= 0:
                    want[:, pg.table[b, to // 16], :, to % 16] = old[name][:, pg.table[b, fr // 16], :, fr % 16]
        assert torch.equal(getattr(pg, name).view(torch.uint8), want)


# ------------------------------------------------------------- E4M3 rounding
def test_e4m3_rows_are_divided_by_their_scale():
    """The stored byte is the quotient's, not that of a product with 1 / scale: scales of the form
    largest / 448, as a calibration gives them, put many quotients on the middle between two codes."""
    mx = lib()
    mant = (torch.arange(128, dtype=torch.int32) + 0x3F80).to(torch.int16).view(BF16)  # [1, 2)
    scales = (mant.float() / 448).cuda()
    heads = 128
    x = torch.stack([mant, -mant * 2 ** -3, mant * 2 ** -9, mant * 8]).cuda()  # [4 tokens, 128]
    pool = torch.zeros(2, heads, 16, 128, dtype=torch.uint8, device="cuda").view(E4M3)
    vpool = torch.zeros(2, heads, 16, 128, dtype=torch.uint8, device="cuda").view(E4M3)
    cache = mx.KVCache(pool, vpool, scales, scales)
    qkv = torch.cat([x[:, None], x[:, None].expand(4, 2 * heads, 128)], 1).reshape(4, -1).contiguous()
    batch = mx.KVBatch(ints([0, 4]), ints([4]), ints([[1]]), tokens=4, max_q=4, max_seq=4)
    mx.rope_append(qkv, 1, None, cache, batch)
    want = (x.float()[None] / scales[:, None, None]).clamp(-448, 448).to(E4M3)  # [heads, 4, 128]
    for got in (pool, vpool):
        assert torch.equal(got.view(torch.uint8)[1, :, :4], want.view(torch.uint8))


# ------------------------------------------------------------ long positions
@pytest.mark.parametrize("near", [0, 2 ** 17, 2 ** 24, 2 ** 28, 2 ** 31 - 70])
def test_angles_at_long_positions(near):
    """Error of an angle: 2^-22 of a turn up to position 2^24, and 2^-47 of position * inv_freq beyond."""
    mx = lib()
    pos = [near + 7 * i for i in range(9)] + [-(near + 5 * i) for i in range(9)]
    inv, _ = mx.rope_frequencies(128)
    inv[0] = 0.9999999  # products that are not whole
    pg = Paged(1, [18], 1, 128, 32)
    qkv = torch.ones(18, 4 * 128, dtype=BF16, device="cuda")
    q = mx.rope_append(qkv, 2, inv, pg.cache(mx), pg.batch(mx, [18]), positions=ints(pos))
    p64 = torch.tensor(pos, dtype=torch.float64, device="cuda")
    ang = p64[:, None] * inv.double()
    c, s = torch.cos(ang), torch.sin(ang)
    ref = torch.cat([c - s, s + c], 1)
    turns = 2 ** -22 + (p64.abs()[:, None] * inv.double() * 2 ** -47)
    # An angle off by t turns moves cos - sin by at most sqrt(2) 2 pi t; sines are good to 2^-21; one bf16 rounding.
    slack = (turns * 2 * math.pi * math.sqrt(2) + 2 ** -20).repeat(1, 2)
    for h in range(2):
        check(q[:, h], ref, ref.abs() * 2 ** -8 + slack, f"positions near {near}")


# ------------------------------------------------------------- a whole step
def test_a_step_captured_once():
    """Room for the new tokens, their page copies, norm, rotary positions with the cache write, attention and accept
    in one graph: replays while lengths, pages and accepted counts change give what the calls give one by one."""
    mx = lib()
    heads, kv, dim, page, new, n, width = 4, 2, 64, 16, 4, 3, 12
    hidden, qkv_width = heads * dim, (heads + 2 * kv) * dim
    inv, factor = mx.rope_frequencies(dim)
    same, grow = ints(list(range(n))), ints([new] * n)
    start = ints([i * new for i in range(n + 1)])

    class Step:
        def __init__(self):
            g = gen(5)
            pool = torch.zeros(2, 2, 60, kv, page, dim, dtype=BF16, device="cuda")  # K and V, two layers
            self.cache, self.pool = mx.KVCache(pool[0], pool[1]), pool
            self.layers = [self.cache.layer(i) for i in range(2)]
            self.table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
            self.lens, self.keep = ints([0] * n), ints([0] * n)
            self.x, self.res, self.w = randn(g, n * new, hidden), randn(g, n * new, hidden), randn(g, hidden)
            self.qkv = randn(g, n * new, qkv_width)
            self.path, self.took = torch.zeros(n, new, dtype=torch.int32, device="cuda"), ints([1] * n)
            # The table and lengths that calls read: every step's new ones are copied there.
            self.batch = mx.KVBatch(start, self.lens, self.table, tokens=n * new, max_q=new, max_seq=width * page)

        def run(self):
            table, lens, copies, self.info = mx.cache_update(self.cache, self.table, self.lens, same, self.keep, grow)
            mx.cache_copy(self.cache, copies)
            self.table.copy_(table)
            self.lens.copy_(lens)
            r = self.res
            for layer in self.layers:
                y, r = mx.residual_norm(self.x, r, self.w)
                q = mx.rope_append(self.qkv, heads, inv, layer, self.batch, factor=factor)
                a = mx.attention(q, layer, self.batch)
                r = a.view(n * new, hidden) + y
            self.out = r
            self.keep.copy_(mx.cache_accept(self.cache, self.batch, self.path, self.took))

    plain, caught = Step(), Step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        caught.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught.run()
    for s in (caught,):  # as at the start
        s.table.fill_(-1)
        s.lens.zero_()
        s.keep.zero_()
        s.pool.zero_()
    for turn in range(9):
        g = gen(100 + turn)
        fresh = randn(g, n * new, qkv_width), randn(g, n * new, hidden)
        order = torch.rand(n, new, generator=g, device="cuda").argsort(1).to(torch.int32)
        took = torch.randint(1, new + 1, (n,), generator=g, device="cuda").to(torch.int32)
        for s in (plain, caught):
            s.qkv.copy_(fresh[0])
            s.x.copy_(fresh[1])
            s.path.copy_(order)
            s.took.copy_(took)
        plain.run()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("table", "lens", "keep", "info", "out", "pool"):
            a, b = getattr(plain, name), getattr(caught, name)
            assert torch.equal(a, b), f"step {turn}: {name}"
        assert plain.info[1].item() == 0 and torch.isfinite(plain.out.float()).all()
    assert int(plain.keep.min()) >= 9
