"""The step's norms, rotary positions with the cache write, and page
bookkeeping against plain float64 / whole-number forms."""
import math

import pytest
import torch

from gpu_cases import Guarded, lib
from step_cases import E4M3, Paged, check, gen, ints, nan_pool, pages_for, randn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


# -------------------------------------------------------------------- norms
def norm64(z, layer, eps):
    if layer:
        z = z - z.mean(1, keepdim=True)
    return z / torch.sqrt((z * z).mean(1, keepdim=True) + eps)


@pytest.mark.parametrize("t,n", [(1, 1), (3, 7), (1, 8), (5, 64), (2, 1000), (4, 7168), (3, 1023), (2, 8200), (2, 9001),
                                 (2, 16392), (1, 32768), (300, 520)])
@pytest.mark.parametrize("kind,post,gate", [("rms", False, None), ("rms", True, "channel"), ("layer", True, "token"),
                                            ("layer", False, "strided")])
def test_residual_norm(t, n, kind, post, gate):
    mx = lib()
    g = gen(n + t)
    x, res = randn(g, t, n), randn(g, t, n) * 2
    w, pw = randn(g, n), randn(g, n) if post else None
    layer = kind == "layer"
    bias, pb = (randn(g, n), randn(g, n) if post else None) if layer else (None, None)
    gt = {None: None, "channel": randn(g, n), "token": randn(g, t, n),
          "strided": randn(g, t, n + 8)[:, :n]}[gate]
    y, r = Guarded((t, n), BF16), Guarded((t, n), BF16)
    mx.residual_norm(x, res, w, post_weight=pw, post_bias=pb, gate=gt, bias=bias, scale=0.5, eps=1e-5,
                     weight_offset=1.0, kind=kind, out=y.t, residual_out=r.t)
    y.check("y")
    r.check("r")
    u = x.double()
    if post:
        u = norm64(u, layer, 1e-5) * (pw.double() + 1)
        if pb is not None:
            u = u + pb.double()
    if gt is not None:
        u = u * gt.double()
    rr = res.double() + 0.5 * u
    # One rounding to bf16 (8 significant bits: half a step is 2^-8 of the value); the fp32 steps before it are
    # good to a few 2^-24 of the terms' size, 2^-18 of which is allowed.
    check(r.t, rr, rr.abs() * 2 ** -8 + 2 ** -18 * (res.double().abs() + u.abs()), "residual")
    z = norm64(rr, layer, 1e-5) * (w.double() + 1)
    size = z.abs()
    if layer:  # centring cancels: what is lost is of the size of the row's mean over its spread
        spread = (rr - rr.mean(1, keepdim=True)).pow(2).mean(1, keepdim=True).add(1e-5).sqrt()
        lost = 2 ** -20 * (rr.abs().amax(1, keepdim=True) + u.abs().amax(1, keepdim=True)) / spread
        size = size + lost * 2 ** 18 * (w.double() + 1).abs()
    if bias is not None:
        z = z + bias.double()
        size = size + bias.double().abs()
    # The norm's own factor carries the error of r, at most 2^-20 of the row's largest terms over its rms.
    rms = rr.pow(2).mean(1, keepdim=True).add(1e-5).sqrt()
    drift = 2 ** -20 * (res.double().abs() + u.abs()).amax(1, keepdim=True) / rms * (w.double() + 1).abs()
    check(y.t, z, z.abs() * 2 ** -8 + 2 ** -18 * size + drift, "y")


def test_residual_norm_in_place_and_row_of_zeros():
    mx = lib()
    g = gen(1)
    x, res, w = randn(g, 6, 256), randn(g, 6, 256), randn(g, 256)
    x[2], res[2] = 0, 0
    y, r = mx.residual_norm(x, res, w)
    assert torch.equal(y[2], torch.zeros_like(y[2]))
    x2, res2 = x.clone(), res.clone()
    mx.residual_norm(x2, res2, w, out=x2, residual_out=res2)
    assert torch.equal(x2, y) and torch.equal(res2, r)


# ------------------------------------------------------------------- rotary
def rope_ref(x, pos, inv_freq, rotary, interleaved, factor):
    """x float64 [t, h, d]"""
    o = x.clone()
    half = rotary // 2
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        ang = pos.double() * inv_freq[j].double()
        c, s = (torch.cos(ang) * factor)[:, None], (torch.sin(ang) * factor)[:, None]
        o[..., a] = x[..., a] * c - x[..., b] * s
        o[..., b] = x[..., a] * s + x[..., b] * c
    return o


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,kv,dim,rotary,page", [(7, 1, 128, 128, 16), (4, 4, 64, 32, 32), (6, 2, 128, 36, 64),
                                                      (3, 1, 64, 2, 16), (8, 2, 64, 0, 128), (56, 8, 128, 96, 64)])
def test_rope_append(dtype, interleaved, heads, kv, dim, rotary, page):
    mx = lib()
    news, lens = [3, 0, 17, 1], [3, 40, 50, 131]
    pg = Paged(dim + rotary, [0] * 4, kv, dim, page, dtype, spare=sum(pages_for(n, page) for n in lens) + 2,
               width=pages_for(131, page))
    order = torch.randperm(pg.num_pages, generator=gen(4), device="cuda").to(torch.int32)
    at = 0
    for b, n in enumerate(lens):
        pg.table[b, :pages_for(n, page)] = order[at:at + pages_for(n, page)]
        at += pages_for(n, page)
    g = gen(rotary)
    t = sum(news)
    wide = randn(g, t, (heads + 2 * kv) * dim + 16)
    qkv = wide[:, :-16]
    if dtype == E4M3:
        qkv[0, heads * dim:] *= 1e4  # saturates
    inv, amp = (mx.rope_frequencies(rotary, scaling="ramp", factor=4.0, trained=2048) if rotary else (None, 1.0))
    cache, batch = pg.cache(mx), pg.batch(mx, news, lens=lens)
    for positions in (None, ints([100000 + 17 * i for i in range(t)])):
        pg.kp.view(torch.uint8).fill_(0xFF)
        pg.vp.view(torch.uint8).fill_(0xFF)
        q = Guarded((t, heads, dim), BF16)
        mx.rope_append(qkv, heads, inv, cache, batch, interleaved=interleaved, positions=positions, factor=amp, out=q.t)
        q.check("q")
        idx = torch.cat([torch.arange(n - m, n) for m, n in zip(news, lens)]).cuda()
        pos = idx if positions is None else positions
        x = qkv.double().view(t, heads + 2 * kv, dim)
        ref = x.clone()
        if rotary:
            ref[:, :heads + kv] = rope_ref(x[:, :heads + kv], pos, inv, rotary, interleaved, amp)
        # Rounding to bf16, and sines and cosines good to 2^-21 (2^-19 allowed).
        size = x.abs().amax(2, keepdim=True) * 2 ** -19
        check(q.t, ref[:, :heads], ref[:, :heads].abs() * 2 ** -8 + size[:, :heads] * 2, "q")
        req = torch.cat([torch.full((m,), b) for b, m in enumerate(news)]).cuda()
        page_ids, rows = pg.table[req, idx // page].long(), idx % page
        for pool, scale, first in ((pg.kp, pg.k_scale, heads), (pg.vp, pg.v_scale, heads + kv)):
            want, slack = ref[:, first:first + kv], size[:, first:first + kv] * 2
            if dtype == E4M3:
                want = (want / scale.double()[:, None]).clamp(-448, 448)
                slack = slack / scale.double()[:, None]
                got = pool.view(torch.uint8)[page_ids, :, rows].view(E4M3)
                # 3 bits of fraction: half a step is 2^-4 of the value, 2^-10 among the subnormals.
                bound = want.abs() * 2 ** -4 + 2 ** -10 + slack
            else:
                got, bound = pool[page_ids, :, rows], want.abs() * 2 ** -8 + slack
            check(got.float(), want, bound, "cache")
            # Nothing else was written.
            left = pool.view(torch.uint8).clone()
            left[page_ids, :, rows] = 0xFF
            assert bool((left == 0xFF).all())


def test_rope_append_skips_missing_pages_and_rows_without_a_request():
    mx = lib()
    pg = Paged(1, [0], 1, 64, 16, spare=3, width=2)
    pg.table[0] = ints([1, 99])  # the second page does not exist
    cache = pg.cache(mx)
    batch = mx.KVBatch(ints([0, 4]), ints([18]), pg.table, tokens=6, max_q=4, max_seq=18)
    qkv, out = randn(gen(1), 6, 4 * 64), torch.full((6, 2, 64), math.nan, dtype=BF16, device="cuda")
    mx.rope_append(qkv, 2, mx.rope_frequencies(64)[0], cache, batch, out=out)
    torch.cuda.synchronize()
    assert torch.isfinite(out[:4].float()).all() and torch.isnan(out[4:].float()).all()
    wrote = torch.isfinite(pg.kp.float()).all(-1)[:, 0]
    assert wrote.nonzero().tolist() == [[1, 14], [1, 15]]


@pytest.mark.parametrize("scaling", [None, "linear", "base", "ramp"])
def test_rope_frequencies(scaling):
    mx = lib()
    freq, amp = mx.rope_frequencies(64, base=10000.0, scaling=scaling, factor=8.0, trained=4096, device="cpu")
    plain = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    ratio = freq.double() / plain
    assert freq.dtype == torch.float32 and freq.shape == (32,)
    if scaling is None:
        assert torch.allclose(ratio, torch.ones(32, dtype=torch.float64), rtol=1e-6)
    elif scaling == "linear":
        assert torch.allclose(ratio, torch.full((32,), 0.125, dtype=torch.float64), rtol=1e-6)
    else:  # the fastest pair stays, the slowest is stretched by the factor, no pair's ratio rises
        assert abs(ratio[0] - 1) < 1e-6 and abs(ratio[-1] - 0.125) < 1e-6
        assert bool((ratio[1:] <= ratio[:-1] + 1e-6).all())
    assert amp == (0.1 * math.log(8.0) + 1 if scaling == "ramp" else 1.0)


# -------------------------------------------------------------------- pages
def update_ref(table, lens, parent, keep, grow, pages, page):
    width = len(table[0])
    base, want, mine = [], [], []
    for i, p in enumerate(parent):
        old = min(max(lens[p], 0), width * page) if 0 <= p < len(lens) else 0
        b = old if keep is None else min(max(keep[i], 0), old)
        base.append(b)
        want.append(min(b + max(grow[i], 0), width * page))
        mine.append([table[p][c] if 0 <= table[p][c] < pages else -1 for c in range(pages_for(b, page))])
    holds, writes = {}, {}
    for i, row in enumerate(mine):
        for e in row:
            holds.setdefault(e, []).append(i)
        if base[i] % page and want[i] > base[i] and row[-1] >= 0:
            writes.setdefault(row[-1], []).append(i)
    free = [p for p in range(pages) if p not in holds]
    count, asked = len(free), 0
    tables, out_lens, copies = [], [], []
    for i, row in enumerate(mine):
        copy = False
        if base[i] % page and want[i] > base[i] and row[-1] >= 0:
            w = writes[row[-1]]
            copy = not (len(w) == len(holds[row[-1]]) and w[0] == i)
        need = int(copy) + pages_for(want[i], page) - len(row)
        asked += need
        got, free = free[:need], free[need:]
        new, moved = list(row), [-1, -1, 0]
        if copy and got:
            moved = [row[-1], got[0], base[i] % page]
            new[-1] = got[0]
            got = got[1:]
        if copy and moved[0] < 0:
            out_lens.append(base[i])
        else:
            new += got
            out_lens.append(min(want[i], len(new) * page))
        tables.append(new + [-1] * (width - len(new)))
        copies.append(moved)
    return tables, out_lens, copies, [len(free), asked - (count - len(free))]


def forked(seed, sequences, pages, width, page):
    """A state that two rounds of random forks, cuts and growth leave behind, from update_ref itself."""
    g = torch.Generator().manual_seed(seed)

    def rnd(lo, hi, n=sequences):
        return torch.randint(lo, hi, (n,), generator=g).tolist()

    table, lens = [[-1] * width for _ in range(sequences)], [0] * sequences
    args = None
    for turn in range(4):
        parent = rnd(-1, sequences) if turn else list(range(sequences))
        keep = None if turn == 1 else rnd(0, width * page)
        grow = rnd(-2, 2 * page + 3)
        args = (table, lens, parent, keep, grow)
        if turn < 3:
            table, lens, _, _ = update_ref(*args, pages, page)
    return args


@pytest.mark.parametrize("seed,sequences,pages,width,page", [
    (1, 4, 64, 8, 16), (2, 32, 400, 12, 16), (3, 32, 90, 12, 32), (4, 1, 3, 2, 16), (5, 200, 2500, 12, 64),
    (6, 1300, 6000, 6, 16), (7, 16, 20, 6, 16), (8, 3, 70000, 40, 16), (9, 64, 300, 5, 128)])
def test_cache_update(seed, sequences, pages, width, page):
    """Forks, cuts, growth and pools that run short, against the rule written out."""
    mx = lib()
    table, lens, parent, keep, grow = forked(seed, sequences, pages, width, page)
    ref = update_ref(table, lens, parent, keep, grow, pages, page)
    pool = torch.empty(pages, 1, page, 64, dtype=BF16, device="cuda")
    wide = torch.full((sequences, width + 3), 7, dtype=torch.int32, device="cuda")
    wide[:, :width] = ints(table)
    ws = Guarded((mx.load().mxfp4_cache_workspace_size(sequences, pages),), torch.uint8)
    for _ in range(2):  # the second call finds the first one's workspace
        got = mx.cache_update(mx.KVCache(pool, pool), wide[:, :width], ints(lens), ints(parent),
                              None if keep is None else ints(keep), ints(grow), workspace=ws.t)
        ws.check("workspace")
        for a, b, name in zip(got, ref, ("table", "lens", "copies", "info")):
            assert a.tolist() == b, name


def test_cache_update_frees_everything():
    mx = lib()
    pool = torch.empty(9, 1, 16, 64, dtype=BF16, device="cuda")
    table, lens, copies, info = mx.cache_update(mx.KVCache(pool, pool), ints([[3, 4, -1], [5, -1, -1]]), ints([20, 3]),
                                                ints([-1, 2]), None, ints([0, 0]))
    assert table.tolist() == [[-1] * 3] * 2 and lens.tolist() == [0, 0] and info.tolist() == [9, 0]
    assert copies.tolist() == [[-1, -1, 0]] * 2


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("kv,dim,page,layers", [(2, 64, 16, None), (8, 128, 64, 3), (1, 128, 128, 2)])
def test_cache_copy(dtype, kv, dim, page, layers):
    mx = lib()
    lead = () if layers is None else (layers,)
    both = torch.randint(0, 255, lead + (12, 2, kv, page, dim * (1 if dtype == E4M3 else 2)), dtype=torch.uint8,
                         device="cuda", generator=gen(page))
    before = both.clone()
    k, v = both.view(dtype).unbind(len(lead) + 1)
    copies = [[3, 7, page], [-1, -1, 0], [3, 0, 5], [11, 1, 1], [2, 12, 4], [2, 5, 0]]  # page 12 does not exist
    mx.cache_copy(mx.KVCache(k, v), ints(copies))
    want = before.view(lead + both.shape[len(lead):])
    for s, d, n in copies:
        if s >= 0 and d < 12:
            want[..., d, :, :, :n, :] = before[..., s, :, :, :n, :]
    assert torch.equal(both, want)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("kv,dim,page,layers", [(2, 64, 16, None), (3, 128, 32, 2)])
def test_cache_accept(dtype, kv, dim, page, layers):
    """Paths in any order, entries out of range, more accepted than the path holds, requests without new tokens."""
    mx = lib()
    lens, news = [70, 64, 31, 9, 5], [64, 10, 0, 8, 5]
    pg = Paged(2, lens, kv, dim, page, dtype, layers=layers)
    es = 1 if dtype == E4M3 else 2
    for pool in (pg.kp, pg.vp):
        pool.view(torch.uint8).copy_(torch.randint(0, 255, pool.view(torch.uint8).shape, dtype=torch.uint8,
                                                   device="cuda", generator=gen(3)))
    path = torch.full((5, 64), 999, dtype=torch.int32)
    path[0] = torch.randperm(64, generator=torch.Generator().manual_seed(1))
    path[1, :6] = torch.tensor([0, 2, -3, 9, 10, 5])
    path[3, :8] = torch.tensor([7, 6, 5, 4, 3, 2, 1, 0])
    path[4, :2] = torch.tensor([3, 4])
    took = [64, 6, 3, 100, -1]
    before = {n: getattr(pg, n).view(torch.uint8).clone() for n in ("kp", "vp")}
    out = mx.cache_accept(pg.cache(mx), pg.batch(mx, news), path.cuda(), ints(took))
    assert out.tolist() == [6 + 64, 54 + 6, 31, 1 + 8, 0]
    shape = (layers or 1, pg.num_pages, kv, page, dim * es)
    for name in ("kp", "vp"):
        want, old = before[name].view(shape).clone(), before[name].view(shape)
        for b in range(5):
            first = lens[b] - news[b]
            for i in range(min(max(took[b], 0), news[b])):
                j = int(path[b, i])
                if 0 <= j < news[b]:
                    to, fr = first + i, first + j
                    want[:, pg.table[b, to // page], :, to % page] = old[:, pg.table[b, fr // page], :, fr % page]
        assert torch.equal(getattr(pg, name).view(torch.uint8).view(shape), want)


def test_verify_step_runs_through():
    """Accept, cut back, fork, copy, write and attend: the tokens a forked
    sequence sees are its parent's accepted ones, and the parent keeps its own."""
    mx = lib()
    heads, kv, dim, page = 8, 2, 64, 16
    pg = Paged(12, [37, 20], kv, dim, page, spare=12, width=6)
    cache = pg.cache(mx)
    lens = mx.cache_accept(cache, pg.batch(mx, [8, 4]), ints([[0, 3, 5], [1, 2, 0]]), ints([3, 1]))
    table, lens2, copies, info = mx.cache_update(cache, pg.table, ints([37, 20]), ints([0, 0, 1]), lens[[0, 0, 1]].contiguous(),
                                                 ints([2, 4, 1]))
    mx.cache_copy(cache, copies)
    assert lens.tolist() == [32, 17] and lens2.tolist() == [34, 36, 18] and info[1].item() == 0
    k0, v0 = ([torch.cat([x[:29], x[29:][[0, 3, 5]]]) for x in (pg.k[0], pg.v[0])])
    k1, v1 = ([torch.cat([x[:16], x[16:][[1]]]) for x in (pg.k[1], pg.v[1])])
    pg.lens, pg.table = [34, 36, 18], table
    batch = pg.batch(mx, [2, 4, 1])
    qkv = randn(gen(9), 7, (heads + 2 * kv) * dim)
    q = mx.rope_append(qkv, heads, None, cache, batch)
    new = qkv.double().view(7, heads + 2 * kv, dim)
    pg.k = [torch.cat([a, new[s:e, heads:heads + kv]]) for a, s, e in ((k0, 0, 2), (k0, 2, 6), (k1, 6, 7))]
    pg.v = [torch.cat([a, new[s:e, heads + kv:]]) for a, s, e in ((v0, 0, 2), (v0, 2, 6), (v1, 6, 7))]
    from step_cases import attention_bound, attention_ref
    out = mx.attention(q, cache, batch)
    ref, _, mag = attention_ref(pg, q, dim ** -0.5)
    check(out, ref, attention_bound(ref, mag), "after the fork")
