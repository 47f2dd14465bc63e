"""Every way that quantize_mx loads its rows: at multiples of 32 bytes or of 16
only, by the rows' begin or by their stride, short and long rows, gated or not."""
import pytest
import torch

from chunk_cases import E4M3, elements, product, round_to, scale_exponents, sum_bound
from gpu_cases import Guarded, lib
from step_cases import check, gen, randn

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8

# (values before the row, values between rows' ends and begins): the stride is a multiple of 8, at times not of 16.
PLACES = [(0, 0), (8, 24), (16, 16), (0, 8), (8, 0), (24, 40)]


def rows(g, t, width, before, between):
    buffer = randn(g, t * (width + between) + before + 64)
    return buffer[before:before + t * (width + between)].view(t, width + between)[:, :width]


@pytest.mark.parametrize("before,between", PLACES)
@pytest.mark.parametrize("t,k", [(37, 32), (5, 256), (9, 2048), (4, 2080), (3, 7168), (2, 20480)])
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_rows(form, t, k, before, between):
    """Codes and scales bit by bit."""
    mx = lib()
    x = rows(gen(t * k + before), t, k, before, between)
    assert x.data_ptr() % 16 == 0 and (x.data_ptr() % 32 == 0) == (before % 16 == 0)
    q = Guarded((t, k), E4M3) if form == "e4m3" else Guarded((t, k // 2), U8)
    s = Guarded((t, k // 32), U8)
    mx.quantize_mx(x, form, out=(q.t, s.t))
    q.check("codes")
    s.check("scales")
    e = scale_exponents(x.double(), form)
    assert torch.equal(s.t.int(), (e + 127).int())
    assert torch.equal(elements(q.t), round_to(x.double() / torch.exp2(e.double()).repeat_interleave(32, 1), form))


@pytest.mark.parametrize("before,between", PLACES)
@pytest.mark.parametrize("t,k", [(37, 32), (5, 256), (9, 2048), (4, 2080), (3, 7168), (2, 20480)])
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_gated_rows(form, t, k, before, between):
    """The same bits as of dense rows, which test_quantize_swiglu compares with float64; a few gates far below zero."""
    mx = lib()
    x = rows(gen(t * k + before), t, 2 * k, before, between)
    x[:, 7] = -100.0
    got, want = mx.quantize_mx(x, form, swiglu=True), mx.quantize_mx(x.contiguous().clone(), form, swiglu=True)
    assert torch.equal(got[0].view(U8), want[0].view(U8)) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("t,k", [(1, 128), (70, 512), (300, 2048)])
def test_codes_as_activations_and_weights_at_once(t, k):
    """The rows' products with each other: both operands are one memory."""
    mx = lib()
    q, s = mx.quantize_mx(randn(gen(t), t, k), "e2m1")
    ref, mag = product((q, s), (q, s))
    check(mx.linear_mx(q, s, q, s), ref, ref.abs() * 2.0 ** -8 + sum_bound(k, mag), "x times itself")


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
@pytest.mark.parametrize("t,n", [(1, 32), (700, 2048), (5, 16416)])
def test_norm_of_one_tensor_as_both_inputs(form, t, n):
    """x as residual too, and the sum written over it."""
    mx, g = lib(), gen(t)
    x, w = randn(g, t, n), randn(g, n)
    want = mx.residual_norm_mx(x, x.clone(), w, scale=0.5, format=form)
    got = mx.residual_norm_mx(x, x, w, scale=0.5, format=form, residual_out=x)
    assert got[2] is x and torch.equal(x, want[2])
    assert torch.equal(got[0].view(U8), want[0].view(U8)) and torch.equal(got[1], want[1])
