"""Microscaled activations and their products with MXFP4 weights against
float64 forms."""
import pytest
import torch

from chunk_cases import E4M3, check_codes, elements, product, random_codes, round_to, scale_exponents, sum_bound, values
from gpu_cases import Guarded, lib
from step_cases import check, gen, randn

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8
FORMATS = ["e4m3", "e2m1"]


def guarded_codes(t, k, form):
    q = Guarded((t, k), E4M3) if form == "e4m3" else Guarded((t, k // 2), U8)
    return q, Guarded((t, k // 32), U8)


# ---------------------------------------------------------- quantisation
@pytest.mark.parametrize("t,k", [(1, 32), (3, 64), (1, 7168), (5, 96), (2, 16384 + 32), (1000, 160), (70, 4096),
                                 (70001, 32), (5003, 96), (999, 2048), (300, 2080)])
@pytest.mark.parametrize("form", FORMATS)
def test_quantize(t, k, form):
    """Elements and scales bit by bit: x is bf16, its quotient by a power of two exact."""
    mx = lib()
    g = gen(t + k)
    x = randn(g, t, k, dtype=torch.float32) * torch.exp2(torch.randint(-40, 40, (t, k // 32), generator=g, device="cuda")
                                                         .float()).repeat_interleave(32, 1)
    x = x.to(BF16)
    q, s = guarded_codes(t, k, form)
    mx.quantize_mx(x, form, out=(q.t, s.t))
    q.check("codes")
    s.check("scales")
    e = scale_exponents(x.double(), form)
    assert torch.equal(s.t.int(), (e + 127).int())
    z = x.double() / torch.exp2(e.double()).repeat_interleave(32, 1)
    assert torch.equal(elements(q.t), round_to(z, form))


@pytest.mark.parametrize("form", FORMATS)
def test_quantize_every_bf16(form):
    """Every finite bf16 number as the largest of its block, next to smaller ones, ties and both zeros."""
    mx = lib()
    bits = torch.arange(0, 0x7f80, device="cuda", dtype=torch.int32).to(torch.int16).view(BF16)
    part = torch.cat([torch.tensor([1.0, -1.0, 0.0, -0.0], device="cuda"), torch.arange(1, 29, device="cuda") / 28])
    x = (bits.double()[:, None] * part.double()).to(BF16)
    x = torch.where(x.abs() > bits[:, None], bits[:, None], x)
    q, s = mx.quantize_mx(x, form)
    e = scale_exponents(x.double(), form)
    assert torch.equal(s.int(), (e + 127).int())
    z = round_to(x.double() / torch.exp2(e.double()).repeat_interleave(32, 1), form)
    assert torch.equal(elements(q), z)
    got = q.view(U8) if form == "e4m3" else torch.stack((q & 15, q >> 4), -1).flatten(1)
    assert torch.equal(got >> (7 if form == "e4m3" else 3), torch.signbit(x).to(U8))  # zeros keep their sign


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantize_not_finite(form, bad):
    mx = lib()
    x = randn(gen(3), 4, 128)
    good = mx.quantize_mx(x, form)
    x[1, 37], x[3, 127] = bad, bad
    q, s = mx.quantize_mx(x, form)
    hit = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[3, 3] = True
    assert torch.equal(s == 255, hit)
    assert torch.equal(s[~hit], good[1][~hit])
    wide = hit.repeat_interleave(32, 1)
    assert torch.equal(elements(q)[~wide], elements(good[0])[~wide])
    if form == "e4m3":
        assert q.float()[wide].isnan().all()


def test_quantize_strided_rows():
    mx = lib()
    x = randn(gen(4), 37, 512)
    for form in FORMATS:
        whole = mx.quantize_mx(x[:, 64:320].contiguous(), form)
        part = mx.quantize_mx(x[:, 64:320], form)
        assert all(torch.equal(a.view(U8), b.view(U8)) for a, b in zip(whole, part))
        narrow = mx.quantize_mx(x[:, 72:328], form)  # an offset of 16 bytes from where 32-byte loads may begin
        assert torch.equal(narrow[1], mx.quantize_mx(x[:, 72:328].contiguous(), form)[1])
        every = mx.quantize_mx(x[::3], form)
        assert torch.equal(every[1], mx.quantize_mx(x[::3].contiguous(), form)[1])


def silu64(a):
    return a * torch.sigmoid(a)


@pytest.mark.parametrize("t,k", [(1, 32), (3, 2048), (129, 96), (33, 18432), (4001, 64)])
@pytest.mark.parametrize("form", FORMATS)
def test_quantize_swiglu(t, k, form):
    mx = lib()
    g = gen(t * k)
    x = randn(g, t, 2 * k) * 3
    x[0, 0], x[0, k] = -200.0, 50.0  # exp overflows: 0
    q, s = guarded_codes(t, k, form)
    mx.quantize_mx(x, form, swiglu=True, out=(q.t, s.t))
    q.check("codes")
    s.check("scales")
    a, b = x.double()[:, :k], x.double()[:, k:]
    z = silu64(a) * b
    # fp32: the exponential is off by (2 + |a|) units of 2^-23, the rest by a few; where exp(-a) passes the
    # range of fp32 the result is 0, and is below 2^-110 of b.
    slack = z.abs() * (8 + a.abs()) * 2.0 ** -23 + b.abs() * 2.0 ** -110
    check_codes(q.t, s.t, z, form, slack, "swiglu")


# ------------------------------------------------------------------ norms
def norm64(z, layer, eps):
    if layer:
        z = z - z.mean(1, keepdim=True)
    return z / torch.sqrt((z * z).mean(1, keepdim=True) + eps)


@pytest.mark.parametrize("t,n", [(1, 32), (3, 96), (5, 1024), (2, 1056), (4, 7168), (700, 2048), (3, 9216), (2, 16416), (1, 32768)])
@pytest.mark.parametrize("kind,post,gate", [("rms", False, None), ("rms", True, "token"), ("layer", True, "channel")])
@pytest.mark.parametrize("form", FORMATS)
def test_residual_norm_mx(t, n, kind, post, gate, form):
    """r has to be residual_norm's own, bit by bit; y, which residual_norm rounds to bf16, goes to its codes unrounded."""
    mx = lib()
    g = gen(n + t)
    x, res, w = randn(g, t, n), randn(g, t, n) * 2, randn(g, n)
    layer = kind == "layer"
    more = dict(post_weight=randn(g, n) if post else None, post_bias=randn(g, n) if post and layer else None,
                gate={None: None, "token": randn(g, t, n), "channel": randn(g, n)}[gate],
                bias=randn(g, n) if layer else None, scale=0.5, eps=1e-5, weight_offset=1.0, kind=kind)
    q, s = guarded_codes(t, n, form)
    r = Guarded((t, n), BF16)
    mx.residual_norm_mx(x, res, w, format=form, out=(q.t, s.t), residual_out=r.t, **more)
    for b, name in ((q, "codes"), (s, "scales"), (r, "residual")):
        b.check(name)
    _, r0 = mx.residual_norm(x, res, w, **more)
    assert torch.equal(r.t, r0)
    u = x.double()
    if post:
        u = norm64(u, layer, 1e-5) * (more["post_weight"].double() + 1)
        if layer:
            u = u + more["post_bias"].double()
    if gate:
        u = u * more["gate"].double()
    rr = res.double() + 0.5 * u
    z = norm64(rr, layer, 1e-5) * (w.double() + 1)
    # What fp32 may lose before the codes, as for residual_norm: 2^-18 of each term, and the row's largest terms over
    # its rms (its spread where centring cancels).
    terms = res.double().abs() + u.abs()
    spread = (rr - rr.mean(1, keepdim=True) if layer else rr).pow(2).mean(1, keepdim=True).add(1e-5).sqrt()
    slack = 2.0 ** -18 * z.abs() + 2.0 ** -20 * terms.amax(1, keepdim=True) / spread * (w.double() + 1).abs() * (3 if layer else 1)
    if layer:
        z = z + more["bias"].double()
        slack = slack + 2.0 ** -18 * more["bias"].double().abs()
    check_codes(q.t, s.t, z, form, slack, "norm")


def test_residual_norm_mx_rows_of_zeros_and_in_place():
    mx = lib()
    g = gen(1)
    x, res, w = randn(g, 6, 256), randn(g, 6, 256), randn(g, 256)
    x[2], res[2] = 0, 0
    x[4, 7] = float("nan")
    for form in FORMATS:
        q, s, r = mx.residual_norm_mx(x, res, w, format=form)
        assert (s[2] == 0).all() and (elements(q)[2] == 0).all()
        assert (s[4] == 255).all() and (s[[0, 1, 2, 3, 5]] != 255).all()
        res2 = res.clone()
        q2, s2, _ = mx.residual_norm_mx(x, res2, w, format=form, residual_out=res2)
        assert torch.equal(res2.view(torch.int16), r.view(torch.int16))
        assert torch.equal(s2, s) and torch.equal(q2.view(U8), q.view(U8))


# --------------------------------------------------------------- products
def weights(g, n, k):
    """Random codes, scales of 2^-5 .. 2^5."""
    return random_codes(g, n, k, "e2m1")


def check_linear(x, w, k):
    mx = lib()
    t, n = x[0].shape[0], w[0].shape[0]
    y = Guarded((t, n), BF16)
    mx.linear_mx(*x, *w, out=y.t)
    y.check("y")
    ref, mag = product(x, w)
    check(y.t, ref, ref.abs() * 2.0 ** -8 + sum_bound(k, mag), f"linear t={t} k={k} n={n}")
    return y.t


@pytest.mark.parametrize("k", [128, 256, 384, 512, 1152, 2048])
@pytest.mark.parametrize("t,n", [(1, 1), (1, 256), (5, 33), (8, 100), (31, 257), (64, 512), (128, 256), (129, 130),
                                 (255, 1000), (257, 64), (300, 770)])
@pytest.mark.parametrize("form", FORMATS)
def test_linear(t, n, k, form):
    g = gen(t + n + k)
    check_linear(random_codes(g, t, k, form), weights(g, n, k), k)


@pytest.mark.parametrize("t,n,k", [(1, 7168, 7168), (16, 7168, 7168), (200, 2048, 18432), (1030, 2304, 1024),
                                   (2500, 9000, 512), (4500, 4100, 256), (40, 40001, 512)])
@pytest.mark.parametrize("form", FORMATS)
def test_linear_large(t, n, k, form):
    """Many tiles a CTA: the ring and both accumulators go round many times."""
    g = gen(t + n + k)
    check_linear(random_codes(g, t, k, form), weights(g, n, k), k)


@pytest.mark.parametrize("form", FORMATS)
def test_linear_single_products(form):
    """One element per row and weight row that is not zero: each product comes out alone, exact in bf16, at its own place."""
    mx = lib()
    t, n, k = 160, 320, 512
    x = torch.zeros(t, k, device="cuda")
    at = torch.arange(t, device="cuda") * 37 % k
    x[torch.arange(t, device="cuda"), at] = (torch.arange(t, device="cuda") % 2 * 2 - 1) * 1.5
    wv = (torch.arange(n, device="cuda")[:, None] + torch.arange(k, device="cuda")) % 7 - 3.0
    w = mx.quantize(wv.contiguous())
    y = mx.linear_mx(*mx.quantize_mx(x.to(BF16), form), *w)
    assert torch.equal(y.double(), (x.double() @ values(*w).T))


@pytest.mark.parametrize("form", FORMATS)
def test_linear_not_finite_rows(form):
    """A NaN block makes its token's outputs NaN and no other's."""
    mx = lib()
    g = gen(11)
    x = randn(g, 150, 640)
    x[7, 600], x[140, 3] = float("nan"), float("inf")
    w = weights(g, 300, 640)
    y = mx.linear_mx(*mx.quantize_mx(x, form), *w)
    bad = torch.zeros(150, dtype=torch.bool, device="cuda")
    bad[7] = bad[140] = True
    assert y[bad].isnan().all() and y[~bad].isfinite().all()


def test_linear_extreme_scales():
    """Scales from 2^-127 to 2^127 on either side: what passes the range of fp32 is infinite, what falls below it 0."""
    mx = lib()
    for form in FORMATS:
        x = torch.ones(4, 128, device="cuda").to(BF16)
        q, s = mx.quantize_mx(x, form)
        wq, ws = mx.quantize(torch.ones(8, 128, device="cuda"))
        s = torch.tensor([0, 100, 250, 254], dtype=U8, device="cuda")[:, None].expand(4, 4).contiguous()
        ws = torch.tensor([0, 10, 127, 150, 200, 253, 254, 4], dtype=U8, device="cuda")[:, None].expand(8, 4).contiguous()
        y = mx.linear_mx(q, s, wq, ws)
        e = s[:, :1].double() + ws[:, 0].double() - 254
        ref = elements(q)[0, 0] * elements(wq)[0, 0] * 128 * torch.exp2(e)
        seen = (ref >= 2.0 ** -120) & (ref < 2.0 ** 127)
        assert torch.equal(y.double()[seen], ref[seen])
        assert y[ref >= 2.0 ** 129].isinf().all() and (y.double()[ref < 2.0 ** -140] == 0).all()


@pytest.mark.parametrize("t,inter,k", [(1, 32, 128), (3, 96, 256), (130, 128, 384), (64, 160, 512), (257, 544, 1152),
                                       (300, 2048, 2048), (1000, 4096, 512), (2100, 4704, 256)])
@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("to", FORMATS)
def test_swiglu(t, inter, k, form, to):
    mx = lib()
    g = gen(t + inter + k)
    x = mx.quantize_mx(randn(g, t, k), form)
    w = mx.quantize(torch.randn(2 * inter, k, generator=g, device="cuda") * 2 * k ** -0.5)
    q, s = guarded_codes(t, inter, to)
    mx.swiglu_mx(*x, *w, format=to, out=(q.t, s.t))
    q.check("codes")
    s.check("scales")
    ref, mag = product(x, w)
    off = sum_bound(k, mag)
    a, b, da, db = ref[:, :inter], ref[:, inter:], off[:, :inter], off[:, inter:]
    z = silu64(a) * b
    # SiLU's slope is at most 1.1; fp32's own part as for quantize_mx.
    slack = 1.1 * da * (b.abs() + db) + a.abs() * db + z.abs() * (8 + a.abs()) * 2.0 ** -23
    check_codes(q.t, s.t, z, to, slack, f"swiglu t={t}")


@pytest.mark.parametrize("form", FORMATS)
def test_block(form):
    """The calls of an FFN block of a chunk, one after another, against the same steps in float64 from the same codes."""
    mx = lib()
    g = gen(5)
    t, k, inter = 77, 512, 640
    x, res, w = randn(g, t, k), randn(g, t, k), randn(g, k) * 0.1 + 1
    w1 = mx.quantize(torch.randn(2 * inter, k, generator=g, device="cuda") * k ** -0.5)
    w2 = mx.quantize(torch.randn(k, inter, generator=g, device="cuda") * inter ** -0.5)
    q, s, r = mx.residual_norm_mx(x, res, w, format=form)
    h = mx.swiglu_mx(q, s, *w1, format=form)
    y = mx.linear_mx(*h, *w2)
    ref, mag = product(h, w2)
    check(y, ref, ref.abs() * 2.0 ** -8 + sum_bound(inter, mag), "y")
    a, mag = product((q, s), w1)
    off = sum_bound(k, mag)
    z = silu64(a[:, :inter]) * a[:, inter:]
    # A bound on the codes' rms (half a step of a normal element over sqrt(3)) does not hold: an element below the least
    # normal one is off by half of a step that does not shrink with it (E2M1: 1/4 of the block's unit). Each one by itself, then.
    slack = 1.1 * off[:, :inter] * (a[:, inter:].abs() + off[:, inter:]) + a[:, :inter].abs() * off[:, inter:] + \
        z.abs() * (8 + a[:, :inter].abs()) * 2.0 ** -23
    check_codes(*h, z, form, slack, "h")
