"""The example's prompt chunks against the same decoder in float64, with the
codes of the definition: the rows behind the last norm, and the K and V rows
that the cache holds afterwards."""
import math
import os
import sys

import pytest
import torch

from chunk_cases import round_to, scale_exponents, values
from gpu_cases import lib

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LAYERS, HEADS, KV, DIM, HIDDEN = 2, 4, 2, 128, 512

# Relative errors by norm.
# K and V of the first layer have one quantisation before them, from inputs that differ by fp32's rounding: next to it two
# roundings to bf16, at most 2^-8 of a value each (the projection's and the rotation's), and codes that fp32 turns to the
# neighbour: of values within 2^-18 of a border between steps of 2^-3 (E2M1: 2^-1) one in 2^14, which by norm is 2^-10.
FIRST = 2 * 2.0 ** -8 + 2.0 ** -10
# From there on the bf16 roundings turn more codes. A step's worth of error d before a quantisation with steps of s turns a
# part d / s of the codes by s each: sqrt(d s) by norm, at most about the quantisation's own error. So the eight
# quantisations of two layers count as independent errors of that size: E4M3 a step of 2^-4 to 2^-3 of a value evenly
# spread, 2^-3.5 / sqrt(12) = 0.026; E2M1, whose steps are 1/2 to 1/4 of a value and 1/2 of a unit below, at most 0.11.
# Twice their sum is allowed: 0.15 and 0.62 (rows that have nothing to do with each other are off by 1.41).
LATER = {"e4m3": 2 * math.sqrt(8) * 0.026, "e2m1": 2 * math.sqrt(8) * 0.11}


def coded(z, form):
    e = scale_exponents(z, form).double()
    unit = torch.exp2(e).repeat_interleave(32, 1)
    return round_to(z / unit, form) * unit


def rotated(x, pos, freq, factor):
    """float64 [tokens, heads, dim], the pairs (j, j + dim / 2)."""
    angle = pos.double()[:, None, None] * freq.double()
    c, s = torch.cos(angle) * factor, torch.sin(angle) * factor
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, a * s + b * c), -1)


def decoder64(model, tokens, form):
    """(rows behind the last norm, [(k, v) of each layer])"""
    def normed(r, w):
        return r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6) * w.double()

    r, pos, kept = model.embed[tokens].double(), torch.arange(len(tokens), device="cuda"), []
    hidden = torch.ones(len(tokens), len(tokens), dtype=torch.bool, device="cuda").triu(1)
    for w in model.layers:
        qkv = coded(normed(r, w["norm1"]), form) @ values(*w["qkv"]).T
        q, k, v = qkv.view(len(tokens), HEADS + 2 * KV, DIM).split((HEADS, KV, KV), 1)
        q, k = (rotated(x, pos, model.inv_freq, model.factor) for x in (q, k))
        kept.append((k, v))
        kk, vv = (x.repeat_interleave(HEADS // KV, 1) for x in (k, v))
        scores = torch.einsum("ihd,jhd->hij", q, kk) * DIM ** -0.5
        a = torch.einsum("hij,jhd->ihd", torch.softmax(scores.masked_fill(hidden, -torch.inf), -1), vv)
        r = r + coded(a.flatten(1), form) @ values(*w["out"]).T
        gate, up = (coded(normed(r, w["norm2"]), form) @ values(*w["up"]).T).chunk(2, 1)
        r = r + coded(gate * torch.sigmoid(gate) * up, form) @ values(*w["down"]).T
    return normed(r, model.norm), kept


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def worst_row(got, want):
    d = (got.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    return float(d.max())


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
@pytest.mark.parametrize("sizes", [[300], [100, 37, 163], [9, 128, 1, 162]])
def test_prompt_against_float64(form, sizes):
    lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import verify_step
    model = verify_step.Decoder(layers=LAYERS, hidden=HIDDEN, heads=HEADS, kv_heads=KV, inter=640, vocab=512)
    tokens = torch.arange(300, device="cuda") * 11 % 512
    cache = model.new_cache(64)
    seq, out, at = verify_step.Sequences(cache, 1, 32), [], 0
    for n in sizes:
        seq.room(n)
        out.append(model.prompt_chunk(tokens[at:at + n], cache, seq.batch(n, 512), form))
        at += n
    rows, kept = decoder64(model, tokens, form)
    pages = seq.table[0, :19].long()
    for i, (k, v) in enumerate(kept):
        for name, pool, want in (("k", cache.k, k), ("v", cache.v, v)):
            got = pool[i][pages].transpose(1, 2).flatten(0, 1)[:300]
            limit = FIRST if i == 0 else LATER[form]
            assert off(got, want) < limit, f"{name} of layer {i}"
            assert worst_row(got, want) < 2 * limit, f"{name} of layer {i}, by rows"
    got = torch.cat(out)
    assert off(got, rows) < LATER[form] and worst_row(got, rows) < 2 * LATER[form]
