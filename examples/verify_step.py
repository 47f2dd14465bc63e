"""A decoder's speculative verify steps, end to end on the library: MXFP4
projections, FFN and LM head next to the norms, rotary positions, paged
attention and page bookkeeping that a step needs.

    python examples/verify_step.py [--layers 4] [--steps 16] [--drafts 3]

Each step takes a sequence's last token and its drafts, runs them through the
model as one chunk, accepts the drafts that agree with the model's own
choices, and moves on: cache_accept keeps the accepted rows, cache_update cuts
the sequence back and makes room for the next chunk. Weights are random; the
drafts are the model's own earlier guesses for the positions ahead.
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import mxfp4_weight_streaming_gb300 as mx  # noqa: E402

BF16 = torch.bfloat16


class Decoder:
    """Random weights of a decoder: per layer an attention block (q, k, v in
    one projection) and a SwiGLU FFN, each behind an RMS norm."""

    def __init__(self, layers=4, hidden=1024, heads=8, kv_heads=2, inter=1024, vocab=4096, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def packed(rows, cols):
            return mx.quantize(torch.randn(rows, cols, generator=g, device=device) * cols ** -0.5)

        def weight(n):
            return (1 + 0.1 * torch.randn(n, generator=g, device=device)).to(BF16)

        self.heads, self.kv_heads, self.dim, self.hidden, self.vocab = heads, kv_heads, hidden // heads, hidden, vocab
        self.embed = torch.randn(vocab, hidden, generator=g, device=device).to(BF16)
        self.layers = [dict(norm1=weight(hidden), norm2=weight(hidden),
                            qkv=packed((heads + 2 * kv_heads) * self.dim, hidden), out=packed(hidden, heads * self.dim),
                            up=packed(2 * inter, hidden), down=packed(hidden, inter)) for _ in range(layers)]
        self.norm, self.head = weight(hidden), packed(vocab, hidden)
        self.inv_freq, self.factor = mx.rope_frequencies(self.dim, device=device)
        self.zero = torch.zeros(64, hidden, dtype=BF16, device=device)

    def new_cache(self, pages, page=16, dtype=BF16, device="cuda"):
        """Pools of all layers."""
        shape = (len(self.layers), pages, self.kv_heads, page, self.dim)
        k, v = (torch.zeros(shape, dtype=BF16, device=device).to(dtype) for _ in range(2))
        scales = [torch.full((self.kv_heads,), 0.02, device=device) for _ in range(2)] if dtype != BF16 else [None, None]
        return mx.KVCache(k, v, *scales)

    def chunk(self, tokens, cache, batch, tree_mask=None):
        """Logits bf16 [tokens, vocab] of a step's new tokens (int64), whose K
        and V go to the cache."""
        r = self.embed[tokens]
        x = self.zero[:r.shape[0]]  # what the block before left to add: nothing
        views = [cache.layer(i) for i in range(len(self.layers))]
        ws = mx.attention_workspace(self.heads, views[0], batch)
        for w, kv in zip(self.layers, views):
            y, r = mx.residual_norm(x, r, w["norm1"])
            q = mx.rope_append(mx.linear(y, *w["qkv"]), self.heads, self.inv_freq, kv, batch, factor=self.factor)
            a = mx.attention(q, kv, batch, tree_mask=tree_mask, workspace=ws)
            y, r = mx.residual_norm(mx.linear(a.view(len(tokens), -1), *w["out"]), r, w["norm2"])
            x = mx.ffn(y, *w["up"], *w["down"])
        y, _ = mx.residual_norm(x, r, self.norm)
        return mx.linear(y, *self.head)


class Sequences:
    """Sequences of a cache between steps: their pages and lengths."""

    def __init__(self, cache, count, width, device="cuda"):
        self.cache = cache
        self.table = torch.full((count, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(count, dtype=torch.int32, device=device)  # with the new tokens, once there is room
        self.same = torch.arange(count, dtype=torch.int32, device=device)

    def room(self, new, keep=None, parent=None):
        """Cuts to keep (all: None), continues `parent` (by default each its own) and makes room for `new` tokens each."""
        parent = self.same if parent is None else parent
        grow = torch.full_like(parent, new)
        self.table, self.lens, copies, info = mx.cache_update(self.cache, self.table, self.lens, parent, keep, grow)
        mx.cache_copy(self.cache, copies)
        self.same = torch.arange(parent.numel(), dtype=torch.int32, device=parent.device)
        return info

    def batch(self, new, max_seq):
        n = self.lens.numel()
        start = torch.arange(n + 1, dtype=torch.int32, device=self.lens.device) * new
        return mx.KVBatch(start, self.lens, self.table, tokens=n * new, max_q=new, max_seq=max_seq)


def generate(model, prompt, steps, drafts=3, pages=256, page=16, dtype=BF16):
    """Greedy continuation of one prompt (a list of tokens) by verify steps of
    1 + drafts tokens; returns (tokens, accepted drafts per step)."""
    cache = model.new_cache(pages, page, dtype)
    seq = Sequences(cache, 1, pages)
    bound = pages * page
    dev = seq.table.device
    for t in range(0, len(prompt) - 1, 8):  # the prompt in chunks of up to 8 (the FFN's limit)
        part = prompt[t:min(t + 8, len(prompt) - 1)]
        seq.room(len(part))
        model.chunk(torch.tensor(part, device=dev), cache, seq.batch(len(part), bound))
    last, guess = torch.tensor([prompt[-1]], device=dev), torch.zeros(drafts, dtype=torch.int64, device=dev)
    out, taken = [], []
    path = torch.arange(1 + drafts, dtype=torch.int32, device=dev)[None]
    keep = None
    for _ in range(steps):
        seq.room(1 + drafts, keep)
        batch = seq.batch(1 + drafts, bound)
        choice = model.chunk(torch.cat([last, guess]), cache, batch).float().argmax(-1)
        agrees = (choice[:-1] == guess).to(torch.int32)
        accepted = agrees.cumprod(0).sum().to(torch.int32).reshape(1)  # drafts, stays on the device
        keep = mx.cache_accept(cache, batch, path, accepted + 1)
        n = int(accepted)
        out += choice[:n + 1].tolist()
        taken.append(n)
        last = choice[n:n + 1]
        guess = torch.cat([choice[n + 1:], choice.new_zeros(n + 1)])[:drafts]
    return out, taken


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--drafts", type=int, default=3)
    a = ap.parse_args()
    model = Decoder(layers=a.layers)
    prompt = [(i * 37 + 11) % model.vocab for i in range(50)]
    generate(model, prompt, 2, a.drafts)
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    tokens, taken = generate(model, prompt, a.steps, a.drafts)
    end.record()
    torch.cuda.synchronize()
    print(f"{len(tokens)} tokens in {a.steps} verify steps of {1 + a.drafts}, {sum(taken)} drafts accepted, "
          f"{begin.elapsed_time(end) / a.steps:.2f} ms a step")
    print(tokens)


if __name__ == "__main__":
    main()
