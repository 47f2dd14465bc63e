"""What is timed of the attention side of a decode / verify step: the norms
around a block, rotary positions with the write into the paged KV cache,
attention of a step's new tokens over that cache, and the bookkeeping of the
cache's pages between steps.

Each operator has a plain form here (elementary torch operations in 32 bits,
rounded once at the end) and the library's own form; `own` picks. `exact`
gives the operators' definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

HIDDEN = 7168  # the dense width of this repository's verify and FFN workloads
HEADS, KV_HEADS, HEAD_DIM = 56, 8, 128  # that width as heads: groups of 7
E4M3_MAX = 448.0


def listed():
    a = dict(op="attention", heads=HEADS, kv_heads=KV_HEADS, head_dim=HEAD_DIM, page=64, dtype="bf16", softcap=0.0,
             window=0, tree=False, ragged=False, strided=False)
    r = dict(op="rope", heads=HEADS, kv_heads=KV_HEADS, head_dim=HEAD_DIM, page=64, dtype="bf16", rotary=128,
             interleaved=False, scaling=1.0)
    c = dict(kv_heads=KV_HEADS, head_dim=HEAD_DIM, page=64, dtype="bf16")
    n = dict(op="norm", n=HIDDEN, post=True, gate="none", kind="rms", scale=1.0)
    return [
        # One user, one token, a short conversation: the smallest call, all latency.
        dict(a, name="attn-decode-b1", batch=1, new=1, ctx=999),
        # Speculative verify for a few users: each a tree of 8 tokens (target and drafts).
        dict(a, name="attn-verify-tree-b8", batch=8, new=8, ctx=4090, ragged=True, tree=True, strided=True),
        # Decode of a full serving batch over an 8-bit cache, lengths as they come.
        dict(a, name="attn-decode-b64-e4m3", batch=64, new=1, ctx=8190, ragged=True, dtype="e4m3"),
        # Verify of one user's 1 target + 3 drafts at the end of a very long document.
        dict(a, name="attn-verify-128k", batch=1, new=4, ctx=131069),
        # Chunks of prompts on layers with a sliding window and capped scores, small pages and heads.
        dict(a, name="attn-chunk-window", batch=4, new=256, ctx=8000, heads=32, kv_heads=8, head_dim=64, page=16,
             window=4096, softcap=50.0, ragged=True),
        # The largest: chunks of two long prompts, the work of a prefill step.
        dict(a, name="attn-chunk-32k", batch=2, new=512, ctx=32000),
        # The rotation and cache write of one verify step.
        dict(r, name="rope-verify-b1", batch=1, new=4, ctx=8188),
        # The same for prompt chunks into an 8-bit cache, half of the head rotated, interleaved, positions stretched.
        dict(r, name="rope-chunk-e4m3", batch=8, new=253, ctx=3700, rotary=64, interleaved=True, scaling=8.0,
             dtype="e4m3"),
        # After a verify step: move the accepted path's rows in every layer, roll back, make room for the next step.
        dict(c, name="cache-accept-b8", op="accept", batch=8, new=8, ctx=300, layers=16),
        # Beams that fork and swap parents: shared pages, copies of the partly filled ones in every layer.
        dict(c, name="cache-fork-b32", op="fork", batch=32, new=1, ctx=1500, layers=24),
        # Norms between two blocks of one verify step (1 target + 3 drafts).
        dict(n, name="norm-verify", tokens=4),
        # The same for prompt chunks, with a gate per token and channel.
        dict(n, name="norm-chunk", tokens=4096, gate="token", scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {c["op"]: max(_cost(x) for x in listed() if x["op"] == c["op"]) for c in listed()}
    op = rng.choice(["attention", "attention", "attention", "rope", "accept", "fork", "norm"])
    while True:
        heads, kv_heads, head_dim = rng.choice([(56, 8, 128), (32, 8, 64), (64, 8, 128), (16, 16, 128), (28, 4, 128),
                                                (40, 8, 64), (12, 2, 128), (16, 1, 128)])
        c = dict(op=op, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=rng.choice([16, 32, 64, 128]),
                 dtype=rng.choice(["bf16", "bf16", "e4m3"]))
        if op == "attention":
            kind = rng.choice(["decode", "verify", "verify", "chunk"])
            c.update(batch=_log(rng, 1, 64 if kind != "chunk" else 8), ctx=_log(rng, 30, 131000),
                     new={"decode": 1, "verify": rng.randint(2, 16), "chunk": _log(rng, 17, 512)}[kind],
                     softcap=rng.choice([0.0, 0.0, 0.0, 30.0]), window=rng.choice([0, 0, 0, 1023, 4096]),
                     tree=kind == "verify" and rng.random() < 0.5, ragged=rng.random() < 0.6,
                     strided=rng.random() < 0.5)
            if c["batch"] * (c["ctx"] + c["new"]) > 550_000:  # memory of the plain form
                continue
        elif op == "rope":
            c.update(batch=_log(rng, 1, 16), new=_log(rng, 1, 300), ctx=_log(rng, 1, 8000),
                     rotary=rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4 * 3]),
                     interleaved=rng.random() < 0.5, scaling=rng.choice([1.0, 1.0, 4.0, 16.0]))
        elif op == "accept":
            c.update(batch=_log(rng, 1, 16), new=rng.randint(2, 32), ctx=_log(rng, 20, 600), layers=rng.randint(1, 16))
        elif op == "fork":
            c.update(batch=_log(rng, 2, 48), new=rng.randint(1, 8), ctx=_log(rng, 20, 3000), layers=rng.randint(1, 24))
        else:
            c = dict(op=op, n=rng.choice([1024, 2048, 4096, 5120, 7168, 8192, 18432, _log(rng, 65, 9000)]),
                     tokens=_log(rng, 1, 4096), post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]),
                     kind=rng.choice(["rms", "rms", "layer"]), scale=rng.choice([1.0, 0.25]))
        # What the plain form has to hold, and what a pass costs, stay within the listed cases.
        if op in ("accept", "fork") and _pool_pages(c) * c["layers"] * kv_heads * c["page"] * head_dim > 600e6:
            continue
        if _cost(c) <= top[op]:
            return c


def _lens(c):
    """Tokens that each request has in the cache before the step."""
    b = c["batch"]
    if not c.get("ragged", c["op"] in ("accept", "fork")):
        return [c["ctx"]] * b
    return [max(1, c["ctx"] - (i * 7919 + 13) % max(1, c["ctx"] // 2)) for i in range(b)]


def _news(c):
    """New tokens of each request in the step."""
    if not c.get("ragged") or c["new"] < 2:
        return [c["new"]] * c["batch"]
    return [max(1, c["new"] - (i * 31) % (c["new"] // 2 + 1)) for i in range(c["batch"])]


def _pages(tokens, page):
    return -(-tokens // page)


def _pool_pages(c):
    if c["op"] == "fork":
        # Every beam's own pages, and as many for the copies and growth.
        return sum(_pages(n, c["page"]) for n in _lens(c)) + 2 * c["batch"] + 8
    return sum(_pages(a + n, c["page"]) for a, n in zip(_lens(c), _news(c))) + 2 * c["batch"] + 3


def _elem(c):
    return 1 if c.get("dtype") == "e4m3" else 2


def _visible(c):
    """(query, key) pairs and cache rows that some query sees, per KV head and query head of a group."""
    pairs = rows = 0
    for a, n in zip(_lens(c), _news(c)):
        w = c["window"] or a + n
        first = max(0, a - w + 1)
        rows += a + n - first
        pairs += sum(min(a + i + 1, w) for i in range(n))
    return pairs, rows


def work(c):
    op = c["op"]
    if op == "attention":
        pairs, rows = _visible(c)
        t = sum(_news(c))
        return {"bytes": 2.0 * rows * c["kv_heads"] * c["head_dim"] * _elem(c) + 4.0 * t * c["heads"] * c["head_dim"],
                "flops": 4.0 * pairs * c["heads"] * c["head_dim"]}
    if op == "rope":
        t = sum(_news(c))
        return {"bytes": float(t * c["head_dim"] * (4 * c["heads"] + 2 * c["kv_heads"] * (2 + _elem(c)))),
                "flops": 3.0 * t * c["rotary"] * (c["heads"] + c["kv_heads"])}
    row = c.get("kv_heads", 0) * c.get("head_dim", 0) * 2 * _elem(c)  # K and V of one token in one layer
    if op == "accept":
        moved = sum(max(0, _accepted(n, i) - 1) for i, n in enumerate(_news(c)))
        table = 8 * sum(_pages(a + n, c["page"]) for a, n in zip(_lens(c), _news(c)))
        return {"bytes": 2.0 * moved * row * c["layers"] + table + 32.0 * c["batch"], "flops": 0.0}
    if op == "fork":
        lens = _lens(c)
        par = _parents(c)
        rows = sum(lens[p] % c["page"] for p in par)
        table = 8 * sum(_pages(lens[p] + c["new"], c["page"]) for p in par)
        return {"bytes": 2.0 * rows * row * c["layers"] + table + 40.0 * c["batch"], "flops": 0.0}
    e = float(c["tokens"]) * c["n"]
    return {"bytes": e * (10 if c["gate"] == "token" else 8) + 2.0 * c["n"] * (1 + c["post"] + (c["gate"] == "channel")),
            "flops": e * 12}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 250)


def _accepted(n, i):
    return 1 + (i * 5 + 2) % n


def _parents(c):
    """Beams of groups of 4: one kept, one twice, one dropped, the last kept."""
    b = c["batch"]
    return [min(b - 1, i - i % 4 + (0, 2, 2, 3)[i % 4]) for i in range(b)]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(c, g, layers=None):
    """Pools of K and V pages with what earlier steps left in them."""
    shape = (_pool_pages(c), c["kv_heads"], c["page"], c["head_dim"])
    if layers:
        shape = (layers,) + shape
    k = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    v = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    if c["dtype"] != "e4m3":
        return k, v, None, None
    ks = torch.empty(c["kv_heads"], device="cuda").uniform_(0.01, 0.05, generator=g)
    vs = torch.empty(c["kv_heads"], device="cuda").uniform_(0.01, 0.05, generator=g)
    return (_e4m3(k, ks), _e4m3(v, vs), ks, vs)


def _e4m3(x, scale):
    return (x.float() / scale[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _table(c, g, lens, spare=0):
    """A block table whose pages lie anywhere in the pool."""
    need = [_pages(n, c["page"]) for n in lens]
    order = torch.randperm(_pool_pages(c), generator=g, device="cuda").to(torch.int32)
    at = torch.tensor(np.concatenate([[0], np.cumsum(need)[:-1]]), device="cuda")
    width = max(need) + spare
    col = torch.arange(width, device="cuda")
    idx = (at[:, None] + col).clamp(max=order.numel() - 1)
    return torch.where(col < _need(need)[:, None], order[idx], -1).to(torch.int32).contiguous()


def _need(need):
    return torch.tensor(need, device="cuda")


def _tree(news, g):
    """Ancestor masks of random draft trees: bit j of a token's word is set where it sees new token j."""
    t, n = len(news), max(news)
    up = torch.rand((t, n), generator=g, device="cuda")
    parent = (up * torch.arange(n, device="cuda").clamp(min=1)).long()  # of token j > 0: one before it
    m = torch.zeros((t, n), dtype=torch.int64, device="cuda")
    m[:, 0] = 1
    for j in range(1, n):
        m[:, j] = m.gather(1, parent[:, j:j + 1])[:, 0] | (1 << j)
    keep = torch.arange(n, device="cuda") < _need(news)[:, None]
    return m[keep].contiguous()


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    s = {"case": c}
    if c["op"] == "norm":
        t, n = c["tokens"], c["n"]
        bf = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
        s.update(x=bf(t, n), residual=bf(t, n) * 3, weight=bf(n) * 0.1 + 1, post=bf(n) * 0.1 + 1 if c["post"] else None,
                 gate={"none": None, "channel": bf(n), "token": bf(t, n)}[c["gate"]],
                 bias=bf(n) * 0.1 if c["kind"] == "layer" else None)
        return s
    lens, news = _lens(c), _news(c)
    total = [a + n for a, n in zip(lens, news)]
    t, h, hk, d = sum(news), c["heads"] if "heads" in c else 0, c["kv_heads"], c["head_dim"]
    s["k"], s["v"], s["k_scale"], s["v_scale"] = _cache(c, g, c.get("layers"))
    s["q_start"] = _ints([0] + list(np.cumsum(news)))
    s["max_q"], s["max_seq"], s["tokens"] = max(news), max(total), t
    if c["op"] == "fork":
        s["seq_lens"] = _ints(lens)
        s["table"] = _table(c, g, lens, spare=_pages(c["new"], c["page"]))
        s["parent"] = _ints(_parents(c))
        s["grow"] = _ints(news)
        s["keep"] = torch.full_like(s["seq_lens"], max(lens))
        return s
    s["seq_lens"] = _ints(total)
    s["table"] = _table(c, g, total, spare=2 if c["op"] == "accept" else 0)
    if c["op"] == "accept":
        order = torch.rand((c["batch"], max(news)), generator=g, device="cuda")
        live = torch.arange(max(news), device="cuda") < _need(news)[:, None]
        took = _need([_accepted(n, i) for i, n in enumerate(news)])
        rank = torch.where(live, order, 2.0).argsort(1).argsort(1)  # a random subset of `took` tokens, ascending
        picked = torch.where(rank < took[:, None], torch.arange(max(news), device="cuda"), max(news))
        s["path"] = picked.sort(1).values.to(torch.int32).contiguous()
        s["n_accept"] = took.to(torch.int32)
        s["parent"] = _ints(list(range(c["batch"])))
        s["grow"] = _ints(news)
        return s
    if c["op"] == "rope":
        s["qkv"] = torch.empty((t, (h + 2 * hk) * d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        j = torch.arange(0, c["rotary"], 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = (10000.0 ** (-j / c["rotary"]) / c["scaling"]).float()
        s["factor"] = 0.1 * math.log(c["scaling"]) + 1.0
        return s
    wide = torch.empty((t, (h + 2 * hk) * d if c["strided"] else h * d), dtype=torch.bfloat16, device="cuda")
    s["q"] = wide.normal_(generator=g)[:, :h * d].unflatten(1, (h, d))
    s["tree"] = _tree(news, g) if c["tree"] else None
    s["scale"] = d ** -0.5
    return s


# ------------------------------------------------------------------- passes
def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _handles(s):
    """What a user's program keeps between calls: the library's views of the cache and of the step."""
    import mxfp4_weight_streaming_gb300 as mx
    s["mx"] = mx
    s["cache"] = mx.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    s["batch"] = mx.KVBatch(s["q_start"], s["seq_lens"], s["table"], tokens=s["tokens"], max_q=s["max_q"],
                            max_seq=s["max_seq"])
    if "q" in s:
        s["ws"] = mx.attention_workspace(s["case"]["heads"], s["cache"], s["batch"])
    if "parent" in s:
        s["ws"] = mx.cache_workspace(s["parent"].numel(), s["cache"].num_pages, s["table"].device)
    return mx


def _own_attention(s):
    mx = s.get("mx") or _handles(s)
    c = s["case"]
    return mx.attention(s["q"], s["cache"], s["batch"], scale=s["scale"], softcap=c["softcap"], window=c["window"],
                        tree_mask=s["tree"], workspace=s["ws"])


def _own_rope(s):
    mx = s.get("mx") or _handles(s)
    c = s["case"]
    q = mx.rope_append(s["qkv"], c["heads"], s["inv_freq"], s["cache"], s["batch"], interleaved=c["interleaved"],
                       factor=s["factor"])
    return {"q": q, "k": s["k"], "v": s["v"]}


def _own_accept(s):
    mx = s.get("mx") or _handles(s)
    lens = mx.cache_accept(s["cache"], s["batch"], s["path"], s["n_accept"])
    table, lens, copies, info = mx.cache_update(s["cache"], s["table"], s["seq_lens"], s["parent"], lens, s["grow"],
                                                workspace=s["ws"])
    return {"table": table, "lens": lens, "copies": copies, "info": info, "k": s["k"], "v": s["v"]}


def _own_fork(s):
    mx = s.get("mx") or _handles(s)
    table, lens, copies, info = mx.cache_update(s["cache"], s["table"], s["seq_lens"], s["parent"], s["keep"],
                                                s["grow"], workspace=s["ws"])
    mx.cache_copy(s["cache"], copies)
    return {"table": table, "lens": lens, "copies": copies, "info": info, "k": s["k"], "v": s["v"]}


def _own_norm(s):
    import mxfp4_weight_streaming_gb300 as mx
    c = s["case"]
    y, r = mx.residual_norm(s["x"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"],
                            bias=s["bias"], scale=c["scale"], kind=c["kind"])
    return {"y": y, "residual": r}


_own = {"attention": _own_attention, "rope": _own_rope, "accept": _own_accept, "fork": _own_fork, "norm": _own_norm}


def _slots(s):
    """Of each new token: its request, cache index, page and row in the page."""
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["q_start"][1:], t, right=True)
    n = s["q_start"].diff()
    at = (s["seq_lens"] - n)[b] + t - s["q_start"][b]
    page = s["case"]["page"]
    return b, at, s["table"][b, at // page].long(), at % page


def _plain_attention(s):
    c = s["case"]
    b, h, hk, d, page = c["batch"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    n, m = s["max_seq"], s["max_q"]
    table = s["table"].clamp(min=0).long()
    width = table.shape[1]
    k = s["k"][table].float().transpose(2, 3).reshape(b, width * page, hk, d)[:, :n]
    v = s["v"][table].float().transpose(2, 3).reshape(b, width * page, hk, d)[:, :n]
    if s["k_scale"] is not None:
        k = k * s["k_scale"][:, None]
        v = v * s["v_scale"][:, None]
    req, at, _, _ = _slots(s)
    i = torch.arange(s["tokens"], device="cuda") - s["q_start"][req]
    q = torch.zeros((b, m, h, d), device="cuda")
    q[req, i] = s["q"].float()
    pos = torch.full((b, m), -1, dtype=torch.long, device="cuda")
    pos[req, i] = at
    j = torch.arange(n, device="cuda")
    see = j <= pos[:, :, None]
    if s["tree"] is not None:
        word = torch.zeros((b, m), dtype=torch.long, device="cuda")
        word[req, i] = s["tree"]
        first = s["seq_lens"] - s["q_start"].diff()
        inside = j - first[:, None]  # index among the new tokens
        bit = (word[:, :, None] >> inside.clamp(0, 63)[:, None]) & 1
        see = torch.where((inside >= 0)[:, None], (bit != 0) & (j < s["seq_lens"][:, None])[:, None], see)
    if c["window"]:
        see = see & (j > pos[:, :, None] - c["window"])
    qg = q.reshape(b, m, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    w = torch.matmul(qg, k.permute(0, 2, 3, 1)) * s["scale"]
    if c["softcap"]:
        w = c["softcap"] * torch.tanh(w / c["softcap"])
    w = w.view(b, hk, h // hk, m, n).masked_fill(~see[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-3e38)
    w = torch.exp(w - top)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(b, hk, -1, n), v.transpose(1, 2)).view(b, hk, h // hk, m, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(b, m, h, d)
    return o[req, i].to(torch.bfloat16)


def _rotate(x, cos, sin, rotary, interleaved):
    r, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = r[..., :rotary // 2], r[..., rotary // 2:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, rest), -1)


def _plain_rope(s):
    c = s["case"]
    h, hk, d = c["heads"], c["kv_heads"], c["head_dim"]
    _, at, page, row = _slots(s)
    x = s["qkv"].float().view(-1, h + 2 * hk, d)
    angle = at[:, None].float() * s["inv_freq"]
    cos, sin = (torch.cos(angle) * s["factor"])[:, None], (torch.sin(angle) * s["factor"])[:, None]
    qk = _rotate(x[:, :h + hk], cos, sin, c["rotary"], c["interleaved"])
    k, v = qk[:, h:], x[:, h + hk:]
    if s["k_scale"] is not None:
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        # rounded to the 8-bit type, then stored by its bytes
        s["k"].view(torch.uint8)[page, :, row] = k.to(torch.float8_e4m3fn).view(torch.uint8)
        s["v"].view(torch.uint8)[page, :, row] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k"][page, :, row] = k.to(torch.bfloat16)
        s["v"][page, :, row] = v.to(torch.bfloat16)
    return {"q": qk[:, :h].to(torch.bfloat16).contiguous(), "k": s["k"], "v": s["v"]}


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _plain_update(s, keep, pages):
    page = s["case"]["page"]
    table, parent, grow = s["table"].long(), s["parent"].long(), s["grow"].long()
    n, width = parent.numel(), table.shape[1]
    seq = torch.arange(n, device="cuda")
    col = torch.arange(width, device="cuda")
    old = torch.where(parent >= 0, s["seq_lens"].long()[parent.clamp(min=0)], 0)
    base = torch.minimum(keep.long().clamp(min=0), old)
    want = (base + grow.clamp(min=0)).clamp(max=width * page)
    kept = (base + page - 1) // page
    mine = torch.where(col < kept[:, None], table[parent.clamp(min=0)], -1)
    dump = torch.where(mine >= 0, mine, pages)
    refs = torch.zeros(pages + 1, dtype=torch.long, device="cuda").scatter_add_(0, dump.view(-1), torch.ones_like(dump.view(-1)))
    writes = (base % page != 0) & (want > base)
    last = torch.where(writes, mine.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0], pages)
    writers = torch.zeros_like(refs).scatter_add_(0, last, torch.ones_like(last))
    lowest = torch.full_like(refs, n).scatter_reduce_(0, last, seq, "amin")
    copy = writes & ~((refs[last] == writers[last]) & (lowest[last] == seq))
    need = copy.long() + (want + page - 1) // page - kept
    off = need.cumsum(0) - need
    free = refs[:pages] == 0
    count = free.sum()
    ids = torch.arange(pages, device="cuda")
    rank = torch.where(free, free.long().cumsum(0) - 1, pages)
    by_rank = torch.full((pages + 1,), -1, dtype=torch.long, device="cuda").scatter_(0, rank, ids)
    by_rank[pages] = -1
    got = torch.minimum((count - off).clamp(min=0), need)
    copied = copy & (got > 0)
    has = kept + got - copied.long()
    lens = torch.where(copy & ~copied, base, torch.minimum(want, has * page))
    pick = off[:, None] + copied[:, None].long() + col - kept[:, None]
    fresh = (col >= kept[:, None]) & (col < has[:, None])
    out = torch.where(fresh, by_rank[pick.clamp(0, pages)], mine)
    dst = by_rank[off.clamp(max=pages)]
    out = torch.where(copied[:, None] & (col == kept[:, None] - 1), dst[:, None], out)
    copies = torch.stack((last, dst, base % page), 1)
    copies = torch.where(copied[:, None], copies, torch.tensor([-1, -1, 0], device="cuda"))
    info = torch.stack((count - got.sum(), need.sum() - got.sum()))
    return out.to(torch.int32), lens.to(torch.int32), copies.to(torch.int32), info.to(torch.int32)


def _plain_accept(s):
    c = s["case"]
    n = s["q_start"].diff()
    first = s["seq_lens"] - n
    i = torch.arange(s["path"].shape[1], device="cuda")
    live = (i < s["n_accept"][:, None]) & (s["path"] < n[:, None])
    b = torch.arange(c["batch"], device="cuda")[:, None].expand_as(live)[live]
    to = (first[:, None] + i)[live].long()
    at = (first[:, None] + s["path"])[live].long()
    page = c["page"]
    for x in (s["k"], s["v"]):
        x = _bytes(x)
        x[:, s["table"][b, to // page].long(), :, to % page] = x[:, s["table"][b, at // page].long(), :, at % page]
    table, lens, copies, info = _plain_update(s, first + s["n_accept"], s["k"].shape[1])
    return {"table": table, "lens": lens, "copies": copies, "info": info, "k": s["k"], "v": s["v"]}


def _plain_fork(s):
    table, lens, copies, info = _plain_update(s, s["keep"], s["k"].shape[1])
    moved = copies[copies[:, 0] >= 0].long()
    row = torch.arange(s["case"]["page"], device="cuda")
    live = row < moved[:, 2:]
    src, dst = moved[:, :1].expand_as(live)[live], moved[:, 1:2].expand_as(live)[live]
    row = row.expand_as(live)[live]
    for x in (s["k"], s["v"]):
        x = _bytes(x)
        x[:, dst, :, row] = x[:, src, :, row]
    return {"table": table, "lens": lens, "copies": copies, "info": info, "k": s["k"], "v": s["v"]}


def _unit(x, kind, eps=1e-6):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def _plain_norm(s):
    c = s["case"]
    u = s["x"].float()
    if s["post"] is not None:
        u = _unit(u, c["kind"]) * s["post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["residual"].float() + c["scale"] * u
    y = _unit(r, c["kind"]) * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.to(torch.bfloat16), "residual": r.to(torch.bfloat16)}


_plain = {"attention": _plain_attention, "rope": _plain_rope, "accept": _plain_accept, "fork": _plain_fork,
          "norm": _plain_norm}


# ------------------------------------------------------- definitions, 64 bits
def exact(case, seed):
    """What `run` returns, from the operators' definitions in 64 bits. None where a value is only moved or counted."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        return _exact_norm(s)
    if c["op"] == "rope":
        return _exact_rope(s)
    if c["op"] == "attention":
        return _exact_attention(s)
    return None


def _exact_norm(s):
    c = s["case"]

    def normed(z):
        mean = z.mean(1, keepdim=True) if c["kind"] == "layer" else torch.zeros_like(z[:, :1])
        return (z - mean) / torch.sqrt((z - mean).pow(2).mean(1, keepdim=True) + 1e-6)

    u = s["x"].double()
    if c["post"]:
        u = normed(u) * s["post"].double()
    if c["gate"] != "none":
        u = s["gate"].double() * u
    r = s["residual"].double() + u * c["scale"]
    y = normed(r) * s["weight"].double() + (s["bias"].double() if s["bias"] is not None else 0.0)
    return {"y": y, "residual": r}


def _exact_rope(s):
    c = s["case"]
    h, hk, d, page, half = c["heads"], c["kv_heads"], c["head_dim"], c["page"], c["rotary"] // 2
    x = s["qkv"].double().view(-1, h + 2 * hk, d)
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(_lens(c), _news(c))]).cuda()
    turn = torch.exp(1j * (pos.double()[:, None] * s["inv_freq"].double())) * s["factor"]  # [t, R/2]
    low = (torch.arange(half) * 2 if c["interleaved"] else torch.arange(half)).cuda()
    high = low + (1 if c["interleaved"] else half)
    z = torch.complex(x[:, :h + hk, low], x[:, :h + hk, high]) * turn[:, None]
    x = x.clone()
    x[:, :h + hk, low], x[:, :h + hk, high] = z.real, z.imag
    k, v = s["k"].double(), s["v"].double()
    table = s["table"].cpu()
    t = 0
    for b, (a, n) in enumerate(zip(_lens(c), _news(c))):
        at = torch.arange(a, a + n)
        p, r = table[b, at // page].long().cuda(), (at % page).cuda()
        for pool, scale, first in ((k, s["k_scale"], h), (v, s["v_scale"], h + hk)):
            rows = x[t:t + n, first:first + hk]
            if scale is not None:
                rows = (rows / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            pool[p, :, r] = rows
        t += n
    return {"q": x[:, :h], "k": k, "v": v}


def _exact_attention(s):
    c = s["case"]
    pairs, _ = _visible(c)
    if 4.0 * pairs * c["heads"] * c["head_dim"] > 6e12:  # over about 20 s in 64 bits
        return None
    h, hk, d, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    out = torch.zeros((s["tokens"], h, d), dtype=torch.float64, device="cuda")
    t = 0
    for b, (a, n) in enumerate(zip(_lens(c), _news(c))):
        pages = s["table"][b, :_pages(a + n, page)].long()
        i = torch.arange(n, device="cuda")[:, None]
        j = torch.arange(a + n, device="cuda")[None]
        see = j <= a + i
        if c["tree"]:
            bits = (s["tree"][t:t + n, None] >> torch.arange(n, device="cuda")) & 1
            see = torch.cat((torch.ones((n, a), dtype=torch.bool, device="cuda"), bits.bool()), 1)
        if c["window"]:
            see = see & (a + i - j < c["window"])
        for kh in range(hk):
            k = s["k"][pages, kh].double().reshape(-1, d)[:a + n]
            v = s["v"][pages, kh].double().reshape(-1, d)[:a + n]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][kh].double(), v * s["v_scale"][kh].double()
            q = s["q"][t:t + n, kh * (h // hk):(kh + 1) * (h // hk)].double()
            w = torch.einsum("igd,jd->gij", q, k) * s["scale"]
            if c["softcap"]:
                w = torch.tanh(w / c["softcap"]) * c["softcap"]
            w = torch.softmax(w.masked_fill(~see, -math.inf), -1)
            w = torch.nan_to_num(w, nan=0.0)
            out[t:t + n, kh * (h // hk):(kh + 1) * (h // hk)] = torch.einsum("gij,jd->igd", w, v)
        t += n
    return out
