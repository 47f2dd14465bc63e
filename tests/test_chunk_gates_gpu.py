"""The gated calls where their values are not ordinary: gates far below zero
next to enormous up values, NaN and infinities."""
import pytest
import torch

from chunk_cases import E4M3, check_codes, elements, values
from gpu_cases import lib
from step_cases import gen, randn

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8
FORMATS = ["e4m3", "e2m1"]


def silu64(a):
    return a * torch.sigmoid(a)


def slack(a, z):
    """fp32's part of SiLU(a) * up = z: the exponential off by (2 + |a|) units of 2^-23, the rest by a few; below
    2^-126 numbers are multiples of 2^-149, or 2^-143 after a division by 64."""
    return z.abs() * (8 + a.abs()) * 2.0 ** -23 + 2.0 ** -142


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("up", [1.0, 2.0 ** 60, 3e38, -3e38])
def test_quantize_gates_far_below_zero(form, up):
    """Each gate alone in its block (the others' up values are 0), so that its own value sets the scale."""
    mx = lib()
    gates = torch.cat([torch.arange(-100, -80, 0.5), torch.tensor([-120.0, -150, -174, -176, -180, -189, -200, -250, -1e4, -1e30])])
    n = len(gates)
    for at in (0, 17, 31):
        x = torch.zeros(n, 64, device="cuda")
        x[:, :32] = -3.0
        x[:, at], x[:, 32 + at] = gates.cuda(), up
        x = x.to(BF16)
        a, b = x.double()[:, :32], x.double()[:, 32:]
        z = silu64(a) * b
        check_codes(*mx.quantize_mx(x, form, swiglu=True), z, form, slack(a, z), f"up {up}")


def test_other_values_of_a_block_do_not_change():
    """What stands beside such a gate comes out with the bits that it has without it."""
    mx, g = lib(), gen(1)
    x = randn(g, 50, 2 * 64) * 3
    x[:, 64 + 5] = 0
    before = mx.quantize_mx(x, swiglu=True)
    x[:, 5] = -95.0
    after = mx.quantize_mx(x, swiglu=True)
    assert torch.equal(before[1], after[1])
    assert torch.equal(elements(before[0]), elements(after[0]))


@pytest.mark.parametrize("form", FORMATS)
def test_swiglu_gates_far_below_zero(form):
    """Sums of two products, exact in fp32, of 16 rows each that are alone in their blocks."""
    mx = lib()
    k, halves = 128, torch.tensor([[4, 1], [4, 1.5], [6, 0], [4, 3], [6, 4], [6, 6], [3, 2], [1, 1]])
    for top in (2.0 ** 3, 2.0 ** 64, 2.0 ** 124):
        inter = 32 * len(halves)
        w = torch.zeros(2 * inter, k, device="cuda")
        rows = torch.arange(len(halves)) * 32 + 7
        w[rows, :2] = -16 * halves.cuda()
        w[inter + rows, 0] = top
        x = torch.zeros(5, k, device="cuda")
        x[:, :2] = 1
        for to in FORMATS:
            q, s = mx.quantize_mx(x.to(BF16), form)
            wq, ws = mx.quantize(w)
            ab = values(q, s) @ values(wq, ws).T
            a, b = ab.chunk(2, 1)
            assert float(a.min()) == -192 and float(b.max()) == top
            z = silu64(a) * b
            check_codes(*mx.swiglu_mx(q, s, wq, ws, format=to), z, to, slack(a, z), f"up {top} to {to}")


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("half", ["gate", "up"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("k", [64, 4096])
def test_quantize_gated_not_finite(form, half, bad, k):
    mx, g = lib(), gen(5)
    x = randn(g, 6, 2 * k)
    good = mx.quantize_mx(x, form, swiglu=True)
    off = 0 if half == "gate" else k
    x[1, off + 37], x[4, off + k - 1] = bad, bad
    q, s = mx.quantize_mx(x, form, swiglu=True)
    hit = torch.zeros(6, k // 32, dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[4, -1] = True
    assert torch.equal(s == 255, hit)
    wide = hit.repeat_interleave(32, 1)
    assert torch.equal(s[~hit], good[1][~hit]) and torch.equal(elements(q)[~wide], elements(good[0])[~wide])
    if form == "e4m3":
        assert q.float()[wide].isnan().all()


@pytest.mark.parametrize("t,inter,k", [(5, 96, 256), (40, 160, 4096), (300, 544, 1152)])
@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("to", FORMATS)
def test_swiglu_not_finite(t, inter, k, form, to):
    """A token with a NaN block: all its outputs. A gate or up row with a NaN scale: that block of every token."""
    mx, g = lib(), gen(6)
    x = randn(g, t, k)
    x[3, k - 1] = float("nan")
    w = torch.randn(2 * inter, k, generator=g, device="cuda") * k ** -0.5
    wq, ws = mx.quantize(w)
    good = mx.swiglu_mx(*mx.quantize_mx(randn(gen(6), t, k), form), wq, ws, format=to)
    ws[40, k // 32 - 1] = 255          # gate row of block 1
    ws[inter + 70, 0] = 255            # up row of block 2
    q, s = mx.swiglu_mx(*mx.quantize_mx(x, form), wq, ws, format=to)
    hit = torch.zeros(t, inter // 32, dtype=torch.bool, device="cuda")
    hit[3] = hit[:, 1] = hit[:, 2] = True
    assert torch.equal(s == 255, hit)
    wide = hit.repeat_interleave(32, 1)
    assert torch.equal(s[~hit], good[1][~hit]) and torch.equal(elements(q)[~wide], elements(good[0])[~wide])
    if to == "e4m3":
        assert q.dtype == E4M3 and q.float()[wide].isnan().all()


# The second is cut over a cluster's CTAs, the third into pairs, the last has many tiles a CTA.
@pytest.mark.parametrize("t,n,k", [(5, 64, 256), (16, 1024, 7168), (300, 512, 2048), (200, 40000, 256)])
@pytest.mark.parametrize("form", FORMATS)
def test_linear_not_finite(t, n, k, form):
    """A NaN block at the begin, in the middle and at the end of k, and a weight row with a NaN scale."""
    mx, g = lib(), gen(7)
    x = randn(g, t, k)
    wq, ws = mx.quantize(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)
    if (t, n, k) == (16, 1024, 7168):
        assert mx.linear_mx_plan(t, k, n, form)["split"] > 1
    want = mx.linear_mx(*mx.quantize_mx(x, form), wq, ws)
    assert want.isfinite().all()
    for i, at in enumerate((0, k // 2 + 3, k - 1)):
        x[i + 1, at] = float("inf") if i == 1 else float("nan")
    ws[n // 2, k // 32 - 1] = 255
    y = mx.linear_mx(*mx.quantize_mx(x, form), wq, ws)
    bad = torch.zeros(t, n, dtype=torch.bool, device="cuda")
    bad[1:4] = bad[:, n // 2] = True
    assert y[bad].isnan().all()
    assert torch.equal(y[~bad].view(torch.int16), want[~bad].view(torch.int16))
    assert U8 is wq.dtype


@pytest.mark.parametrize("t,inter,k", [(4, 2048, 7168), (300, 2048, 2048), (1100, 4096, 512)])
@pytest.mark.parametrize("form", FORMATS)
def test_same_bits_every_time(form, t, inter, k):
    """Norm, gated product and product, one after another, many times."""
    mx, g = lib(), gen(8)
    x, res, w = randn(g, t, k), randn(g, t, k), randn(g, k) * 0.1 + 1
    w1 = mx.quantize(torch.randn(2 * inter, k, generator=g, device="cuda") * k ** -0.5)
    w2 = mx.quantize(torch.randn(k, inter, generator=g, device="cuda") * inter ** -0.5)

    def block():
        q, s, r = mx.residual_norm_mx(x, res, w, format=form)
        h = mx.swiglu_mx(q, s, *w1, format=form)
        return [v.contiguous().view(U8) for v in (q, s, r, *h, mx.linear_mx(*h, *w2))]

    first = block()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(block(), first))
