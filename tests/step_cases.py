"""Shared helpers for the tests of the step's attention side: paged caches
whose unused places hold NaN, and the operators' definitions in float64."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def pages_for(n, page):
    return -(-n // page)


def nan_pool(shape, dtype):
    if dtype == E4M3:
        return torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
    return torch.full(shape, math.nan, dtype=dtype, device="cuda")


def set_rows(pool, page_ids, rows, values):
    """pool[page_ids, :, rows] = values, for 8-bit types by their bytes."""
    if pool.dtype == E4M3:
        pool.view(torch.uint8)[page_ids, :, rows] = values.to(E4M3).view(torch.uint8)
    else:
        pool[page_ids, :, rows] = values.to(pool.dtype)


class Paged:
    """A paged cache with `lens` tokens per sequence, pages at random places
    of the pool, NaN wherever no token lies, -1 or nonsense in unused table
    entries. k, v: per sequence float64 [len, kv_heads, dim] as stored."""

    def __init__(self, seed, lens, kv_heads, dim, page, dtype=torch.bfloat16, spare=2, width=None, interleave=False,
                 layers=None, junk=-1):
        g = gen(seed)
        self.page, self.lens, self.dtype, self.kv_heads, self.dim = page, list(lens), dtype, kv_heads, dim
        need = [pages_for(n, page) for n in lens]
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g, device="cuda").to(torch.int32)
        width = width or max(1, max(need))
        self.table = torch.full((len(lens), width), junk, dtype=torch.int32, device="cuda")
        lead = () if layers is None else (layers,)
        if interleave:  # K and V of a page next to each other
            both = nan_pool(lead + (self.num_pages, 2, kv_heads, page, dim), dtype)
            self.kp, self.vp = both.unbind(len(lead) + 1)
        else:
            self.kp = nan_pool(lead + (self.num_pages, kv_heads, page, dim), dtype)
            self.vp = nan_pool(lead + (self.num_pages, kv_heads, page, dim), dtype)
        self.k_scale = self.v_scale = None
        if dtype == E4M3:
            self.k_scale = torch.rand(kv_heads, generator=g, device="cuda") * 0.02 + 0.005
            self.v_scale = torch.rand(kv_heads, generator=g, device="cuda") * 0.02 + 0.005
        self.k, self.v = [], []
        at = 0
        for b, n in enumerate(lens):
            ids = order[at:at + need[b]]
            self.table[b, :need[b]] = ids
            at += need[b]
            j = torch.arange(n, device="cuda")
            p, r = ids.long()[j // page], j % page
            for kv, pool, scale in ((self.k, self.kp, self.k_scale), (self.v, self.vp, self.v_scale)):
                x = torch.randn(n, kv_heads, dim, generator=g, device="cuda")
                if scale is not None:
                    x = (x / scale[:, None]).clamp(-448, 448).to(E4M3)
                else:
                    x = x.to(dtype)
                layer = pool if layers is None else pool[0]
                if n:
                    set_rows(layer, p, r, x)
                x = x.double()
                kv.append(x if scale is None else x * scale.double()[:, None])

    def cache(self, mx):
        return mx.KVCache(self.kp, self.vp, self.k_scale, self.v_scale)

    def batch(self, mx, news, table=None, lens=None):
        start = [0]
        for n in news:
            start.append(start[-1] + n)
        self.news = list(news)
        self.start = start
        return mx.KVBatch(ints(start), ints(self.lens if lens is None else lens), self.table if table is None else table,
                          tokens=max(start[-1], 1), max_q=max(max(news), 1), max_seq=max(max(self.lens), 1))


def attention_ref(pg, q, scale, softcap=0.0, window=0, tree=None):
    """(out, lse, sum_j p_j |v_j|) in float64 from the definition."""
    t, heads, dim = q.shape
    out = torch.zeros(t, heads, dim, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    lse = torch.full((t, heads), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(pg.news):
        seq = pg.lens[b]
        grp = heads // pg.kv_heads
        for i in range(n):
            row, c = pg.start[b] + i, seq - n + i
            see = torch.zeros(seq, dtype=torch.bool, device="cuda")
            if tree is None:
                see[:max(c + 1, 0)] = True
            else:
                first = max(seq - n, 0)
                see[:first] = True
                word = int(tree[row])
                for j in range(max(n - seq, 0), n):
                    see[seq - n + j] = bool(word >> j & 1)
            if window:
                see &= torch.arange(seq, device="cuda") > c - window
            if not see.any():
                continue
            k = pg.k[b][see].repeat_interleave(grp, 1)
            v = pg.v[b][see].repeat_interleave(grp, 1)
            s = torch.einsum("hd,jhd->hj", q[row].double(), k) * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            lse[row] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            out[row] = torch.einsum("hj,jhd->hd", p, v)
            mag[row] = torch.einsum("hj,jhd->hd", p, v.abs())
    return out, lse, mag


def attention_bound(ref, mag, dtype=torch.bfloat16):
    """The output is rounded to bf16: 8 significant bits, half a step is 2^-8
    of the value. Each probability is rounded to bf16 too (2^-8 of its product
    with v), or with an E4M3 cache to f16 (2^-11); scores are fp32 sums whose
    error of about 1e-5 moves a probability by as much of itself (2^-12 allows
    for many times that)."""
    return ref.abs() * 2 ** -8 + mag * ((2 ** -11 if dtype == E4M3 else 2 ** -8) + 2 ** -12) + 1e-30


def check(got, ref, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} outputs are not finite"
    over = (got - ref).abs() > bound
    if over.any():
        i = tuple(int(x) for x in over.nonzero()[0])
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} outside the bound, first at {i}: "
                             f"{float(got[i])} for {float(ref[i])} (bound {float(bound[i])})")
