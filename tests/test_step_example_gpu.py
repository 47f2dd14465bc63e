"""The example's decoder: a step of several tokens gives the logits that the
same tokens give one at a time, drafts that are right are accepted, and a
forked sequence goes on from its parent's tokens."""
import os
import subprocess
import sys

import pytest
import torch

from gpu_cases import lib

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import verify_step
    return verify_step


def close(a, b, what):
    """Two orders of the same sums: every kernel rounds its outputs to bf16
    (2^-8 each), about 12 of them in a row over two layers, of the logits' rms."""
    a, b = a.double(), b.double()
    off = (a - b).abs().max() / b.square().mean().sqrt()
    assert off < 12 * 4 * 2 ** -8, f"{what}: {float(off)}"


def test_chunk_equals_single_tokens(ex):
    model = ex.Decoder(layers=2, hidden=512, heads=4, kv_heads=2, inter=512, vocab=512)
    tokens = torch.arange(7, 47, device="cuda") * 11 % 512
    one = ex.Sequences(model.new_cache(32), 1, 16)
    logits = []
    for t in range(40):
        one.room(1)
        logits.append(model.chunk(tokens[t:t + 1], one.cache, one.batch(1, 512)))
    logits = torch.cat(logits)
    many = ex.Sequences(model.new_cache(32), 1, 16)
    for t in range(0, 40, 8):
        many.room(8)
        close(model.chunk(tokens[t:t + 8], many.cache, many.batch(8, 512)), logits[t:t + 8], f"tokens {t}..")
    assert int(many.lens) == 40 and int(one.lens) == 40


def test_generate_does_not_depend_on_the_drafts(ex):
    """The tokens of steps with drafts are the model's own single-token choices."""
    model = ex.Decoder(layers=2, hidden=512, heads=4, kv_heads=2, inter=512, vocab=512)
    prompt = [3, 5, 8, 13, 21, 34, 55, 89, 144, 233, 377, 99]
    out, taken = ex.generate(model, prompt, 10, drafts=3)
    assert len(out) == 10 + sum(taken)
    # Teacher-forced check: every token is the argmax, or within rounding of it.
    seq = ex.Sequences(model.new_cache(64), 1, 32)
    every = torch.tensor(prompt + out, device="cuda")
    for t in range(0, len(every) - 1):
        seq.room(1)
        logits = model.chunk(every[t:t + 1], seq.cache, seq.batch(1, 512)).double()[0]
        if t >= len(prompt) - 1:
            gap = logits.max() - logits[every[t + 1]]
            assert gap <= 12 * 4 * 2 ** -8 * logits.square().mean().sqrt() * 2, (t, float(gap))


def test_forks_share_their_parents_tokens(ex):
    model = ex.Decoder(layers=2, hidden=512, heads=4, kv_heads=2, inter=512, vocab=512)
    cache = model.new_cache(24)
    seq = ex.Sequences(cache, 1, 8)
    tokens = torch.arange(21, device="cuda") * 17 % 512
    for t in (0, 7, 14):
        seq.room(7)
        model.chunk(tokens[t:t + 7], cache, seq.batch(7, 128))
    info = seq.room(1, parent=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert info.tolist() == [24 - 1 - 3, 0]  # one full page shared, three of their own
    logits = model.chunk(torch.tensor([9, 9, 400], device="cuda"), cache, seq.batch(1, 128))
    assert torch.equal(logits[0], logits[1]) and not torch.equal(logits[0], logits[2])
    alone = ex.Sequences(model.new_cache(24), 1, 8)
    for t in (0, 7, 14):
        alone.room(7)
        model.chunk(tokens[t:t + 7], alone.cache, alone.batch(7, 128))
    alone.room(1)
    close(logits[2:], model.chunk(torch.tensor([400], device="cuda"), alone.cache, alone.batch(1, 128)), "fork")


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "verify_step.py"), "--layers", "1", "--steps", "3"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "verify steps" in r.stdout
