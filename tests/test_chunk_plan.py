"""How products of many tokens are cut: what the kernel takes for granted of
every plan, over many sizes, on the CPU."""
import itertools
import random

import pytest

import mxfp4_weight_streaming_gb300 as mx

MOST = 232448  # opt-in shared memory of a block


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mxfp4_weight_streaming_gb300 import build
    build.build()
    return mx.load()


def sizes():
    rng = random.Random(1)
    for t, k, n in itertools.product([1, 5, 16, 61, 77, 128, 129, 300, 512, 4096], [128, 512, 2048, 7168, 18432],
                                     [32, 96, 2048, 7168, 129280]):
        yield t, k, n
    for _ in range(1500):
        yield (int(2 ** rng.uniform(0, 16)), 128 * int(2 ** rng.uniform(0, 12)), 32 * int(2 ** rng.uniform(0, 13)))


def check(p, t, k, n, form, swiglu, clusters):
    where = (t, k, n, form, swiglu, p)
    rows = p["token_rows"]
    assert p["width"] % (64 if swiglu else 32) == 0 and 32 <= p["width"] <= 256, where
    assert rows == min(128, -(-t // 8) * 8) and (not p["pair"] or t > 128), where
    assert p["stage_bytes"] == 128 * (rows + p["width"] // (1 + p["pair"])), where
    assert p["stage_bytes"] % 1024 == 0, where  # the swizzle's period
    assert p["scale_bytes"] == (1 + -(-p["width"] // 128)) * 4 * 512, where
    ring = p["ring_slots"] * p["stage_bytes"]
    # Barriers and the alignment of the base take a kilobyte each.
    assert 2 <= p["ring_slots"] <= 16 and 2048 + ring + p["scale_slots"] * p["scale_bytes"] <= p["smem_bytes"] <= MOST, where
    assert p["smem_bytes"] >= 192 * 1024, where
    # A product reads 128 rows of tokens from the begin of a stage, the last one too.
    assert 2048 + (p["ring_slots"] - 1) * p["stage_bytes"] + 128 * 128 <= p["smem_bytes"], where
    # Scales of all stages in the ring fit, or as many groups as there are slots at most.
    assert 3 <= p["scale_slots"] <= 6, where
    cluster = p["split"] * (1 + p["pair"])
    groups = -(-k // 512)
    assert 1 <= p["split"] <= groups and cluster <= 8, where
    outputs = p["width"] // 2 if swiglu else p["width"]
    tiles = -(-t // (128 * (1 + p["pair"]))) * -(-n // outputs)
    if p["split"] > 1:
        # All clusters at once, one tile each; the others' sums lie in the ring.
        assert tiles <= clusters[cluster] and p["ctas"] == tiles * cluster, where
        halves, chunks = 1 + swiglu, outputs // 32
        top = 0
        for c in range(chunks):
            for sender in range(p["split"]):
                if sender != c % p["split"]:
                    place = c // p["split"] * (p["split"] - 1) + sender - (sender > c % p["split"])
                    top = max(top, (place + 1) * halves * 128 * 128)
        assert top <= p["inbox_bytes"] <= ring, where
    else:
        assert p["inbox_bytes"] == 0 and p["ctas"] == cluster * min(tiles, clusters[cluster]), where


GB300 = [0, 152, 76, 46, 36, 28, 23, 15, 15]


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("clusters", [None, [0, 148, 74, 44, 35, 27, 22, 14, 14], [0, 20, 10, 6, 5, 4, 3, 2, 2], [0, 1, 0, 0, 0, 0, 0, 0, 0]])
def test_what_every_plan_keeps(form, swiglu, aligned, clusters):
    for t, k, n in sizes():
        n = n if swiglu or aligned else max(1, n - 31)
        p = mx.linear_mx_plan(t, k, n, form, swiglu, aligned, clusters=clusters)
        check(p, t, k, n, form, swiglu, clusters or GB300)


def test_few_tokens_share_k_and_many_take_pairs():
    assert mx.linear_mx_plan(16, 7168, 7168)["split"] > 1
    assert mx.linear_mx_plan(300, 7168, 2048, swiglu=True)["split"] > 1
    p = mx.linear_mx_plan(4096, 18432, 7168, "e2m1")
    assert p["pair"] == 1 and p["width"] == 256 and p["split"] == 1
    assert mx.linear_mx_plan(61, 7168, 129280)["pair"] == 0


@pytest.mark.parametrize("args,status", [((0, 128, 1), 1), ((1, 0, 1), 1), ((1, 128, 0), 1), ((1, 192, 1), 2),
                                         ((1, (1 << 24) + 128, 1), 2), ((1 << 31, 128, 1), 2), ((1, 128, 1 << 31), 2)])
def test_sizes_that_are_refused(args, status):
    with pytest.raises(mx.Mxfp4Error) as e:
        mx.linear_mx_plan(*args)
    assert e.value.status == status


def test_too_little_shared_memory():
    for most in (20000, 190000):
        with pytest.raises(mx.Mxfp4Error):
            mx.linear_mx_plan(4096, 7168, 7168, max_smem=most)
    with pytest.raises(mx.Mxfp4Error):
        mx.linear_mx_plan(4, 256, 40, swiglu=True)  # inter


def test_more_tiles_than_a_launch_counts():
    """No plan for what a launch would refuse: 2^27 tiles and more."""
    assert mx.linear_mx_plan(1 << 24, 128, 1 << 18)["ctas"] > 0
    with pytest.raises(mx.Mxfp4Error):
        mx.linear_mx_plan(1 << 30, 128, 1 << 30)
