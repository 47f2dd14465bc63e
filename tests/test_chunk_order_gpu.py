"""Weights that the calls right before a product have made: every one reads
what the stream has written by then, whatever runs between the two."""
import itertools

import pytest
import torch

from chunk_cases import random_codes
from gpu_cases import lib
from step_cases import gen, randn

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8
ROUNDS = 12


class Makers:
    """Ways to make E2M1 codes and scales of [n, k], each time others, in the same memory."""

    def __init__(self, n, k):
        mx, g = lib(), gen(n + k)
        self.q, self.s = torch.empty(n, k // 2, dtype=U8, device="cuda"), torch.empty(n, k // 32, dtype=U8, device="cuda")
        self.n, self.k = n, k
        self.x = [randn(g, n, k) for _ in range(ROUNDS)]
        self.r, self.one = torch.empty(n, k, dtype=BF16, device="cuda"), torch.ones(k, dtype=BF16, device="cuda")
        self.x32 = [x.float() for x in self.x]
        self.codes = [mx.quantize_mx(x, "e2m1") for x in self.x]
        self.short = [mx.quantize_mx(randn(g, n, 256)) for _ in range(ROUNDS)]
        self.w1 = mx.quantize(torch.randn(2 * k, 256, generator=g, device="cuda") / 4)
        torch.cuda.synchronize()

    def norm(self, i):
        lib().residual_norm_mx(self.x[i], self.x[i - 1], self.one, format="e2m1", out=(self.q, self.s), residual_out=self.r)

    def swiglu(self, i):
        lib().swiglu_mx(*self.short[i], *self.w1, format="e2m1", out=(self.q, self.s))

    def quantize_mx(self, i):
        lib().quantize_mx(self.x[i], "e2m1", out=(self.q, self.s))

    def quantize(self, i):
        mx = lib()
        rc = mx.mxfp4_quantize(self.x32[i].data_ptr(), self.n, self.k, self.q.data_ptr(), self.s.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
        assert rc == mx.MXFP4_OK

    def other_kernels(self, i):
        """Two of another library."""
        torch.bitwise_xor(self.codes[i][1], 0, out=self.s)
        torch.bitwise_xor(self.codes[i][0], 0, out=self.q)


MAKERS = ["norm", "swiglu", "quantize_mx", "quantize", "other_kernels"]


def unrelated(kind):
    """A call of few CTAs that neither makes nor takes those codes."""
    mx, g = lib(), gen(7)
    if kind == "linear_mx":
        a, w = random_codes(g, 8, 128, "e4m3"), random_codes(g, 64, 128, "e2m1")
        return lambda: mx.linear_mx(*a, *w)
    if kind == "linear":
        a, w = randn(g, 2, 512), random_codes(g, 64, 512, "e2m1")
        torch.cuda.synchronize()
        return lambda: mx.linear(a, *w)
    return lambda: None


def same_as_apart(maker, between, use):
    """`use` right behind the maker (and the calls between) gives what it gives when each waits for the one before."""
    def all_rounds(wait):
        out = []
        for i in range(ROUNDS):
            for step in [lambda: maker(i)] + between:
                step()
                wait()
            out.append(use())
            wait()
        return out

    got = all_rounds(lambda: None)
    want = all_rounds(torch.cuda.synchronize)
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x.contiguous().view(U8), y.contiguous().view(U8))
    assert not torch.equal(want[0][0].view(U8), want[1][0].view(U8))  # each round's weights are others


@pytest.mark.parametrize("between", [(), ("linear_mx",), ("linear",), ("linear_mx", "linear")])
@pytest.mark.parametrize("maker", MAKERS)
@pytest.mark.parametrize("n,k", [(64, 512), (640, 2048)])
def test_products_of_many_tokens(maker, between, n, k):
    mx, g = lib(), gen(3)
    m = Makers(n, k)
    steps = [unrelated(b) for b in between]
    for t, form in itertools.product((5, 200), ("e4m3", "e2m1")):
        x = random_codes(g, t, k, form)
        same_as_apart(getattr(m, maker), steps, lambda: (mx.linear_mx(*x, m.q, m.s),))
        same_as_apart(getattr(m, maker), steps, lambda: mx.swiglu_mx(*x, m.q, m.s))


@pytest.mark.parametrize("between", [(), ("linear_mx",), ("linear",), ("linear_mx", "linear")])
@pytest.mark.parametrize("maker", ["quantize", "quantize_mx"])
@pytest.mark.parametrize("n,k", [(64, 512), (640, 2048), (640, 1056)])
def test_calls_that_read_weights_ahead(maker, between, n, k):
    """mxfp4_linear's three kernels and the FFN's two read weights before they wait for the kernels ahead of them, which
    both packers allow for."""
    mx, g = lib(), gen(4)
    m = Makers(n, k)
    steps = [unrelated(b) for b in between]
    for t in (3, 20):
        x = randn(g, t, k)
        same_as_apart(getattr(m, maker), steps, lambda: (mx.linear(x, m.q, m.s),))
    w2 = mx.quantize(torch.randn(k, n // 2, generator=g, device="cuda"))
    for t in (2, 7):
        x = randn(g, t, k)
        same_as_apart(getattr(m, maker), steps, lambda: (mx.ffn(x, m.q, m.s, *w2),))
