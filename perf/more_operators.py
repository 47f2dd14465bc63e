"""What is timed of a prompt chunk's way through MXFP4 weights: norms and
activations that come out as microscaled codes (MX: blocks of 32 values with
one power-of-two scale; E4M3 or E2M1 elements), and the products of such
codes with MXFP4 weights.

Each operator has a plain form here (elementary torch operations in 32 bits,
rounded once at the end) and the library's own form; `own` picks. `exact`
gives the operators' definitions in 64 bits.
"""
import math

import torch

own = False

HIDDEN, INTER = 7168, 18432  # this repository's verify and FFN workloads
EXPERT = 2048  # its expert width
VOCAB = 129280  # its LM head
QKV = 9216  # that hidden size as 56 query and 2 x 8 KV heads of 128
MOST = {"e4m3": 448.0, "e2m1": 6.0}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    n = dict(op="norm", n=HIDDEN, post=False, gate="none", kind="rms", scale=1.0, format="e4m3")
    q = dict(op="quantize", swiglu=False, strided=False, format="e4m3")
    lin = dict(op="linear", format="e4m3")
    return [
        # The norm before a projection in one verify step (1 target + 3 drafts): all latency.
        dict(n, name="norm-mx-verify", tokens=4),
        # The same for the prompt chunks of a prefill step, norms on both sides of the block and a gate per token.
        dict(n, name="norm-mx-chunk", tokens=4096, post=True, gate="token", scale=0.5),
        # Attention's output for the output projection: an odd number of tokens, rows inside a wider buffer.
        dict(q, name="quantize-attn-1000", t=1001, k=HIDDEN, strided=True),
        # Gate and up of a shared expert, made by an earlier product, for its down projection.
        dict(q, name="quantize-swiglu-2048", t=2048, k=INTER, swiglu=True),
        # A projection for the tokens of 16 requests that decode: the weights' bytes count.
        dict(lin, name="linear-mx-16", t=16, k=HIDDEN, n=HIDDEN),
        # The LM head for the last tokens of a ragged batch.
        dict(lin, name="linear-mx-head-61", t=61, k=HIDDEN, n=VOCAB),
        # The joint projection to q, k and v for one prompt chunk.
        dict(lin, name="linear-mx-qkv-512", t=512, k=HIDDEN, n=QKV),
        # The down projection of a large prefill step, activations in 4 bits.
        dict(lin, name="linear-mx-down-4096-e2m1", t=4096, k=INTER, n=HIDDEN, format="e2m1"),
        # Gate and up of one expert for the tokens that were routed to it.
        dict(op="swiglu", name="swiglu-mx-expert-300", t=300, k=HIDDEN, inter=EXPERT, format="e4m3", to="e4m3"),
        # The largest: gate and up of the dense FFN for a large prefill step.
        dict(op="swiglu", name="swiglu-mx-4096", t=4096, k=HIDDEN, inter=INTER, format="e4m3", to="e4m3"),
        # A whole FFN block of a chunk, norm to output, with 4-bit activations.
        dict(op="block", name="block-1024-e2m1", t=1024, k=HIDDEN, inter=INTER, format="e2m1"),
        # The same for a short chunk with 8-bit activations, of an expert's width.
        dict(op="block", name="block-77", t=77, k=HIDDEN, inter=EXPERT, format="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    op = rng.choice(["norm", "quantize", "linear", "linear", "linear", "swiglu", "swiglu", "block"])
    while True:
        k = rng.choice([HIDDEN, INTER, EXPERT, 4096, 5120, 8192, 128 * _log(rng, 1, 64)])
        n = rng.choice([HIDDEN, QKV, 4096, EXPERT, _log(rng, 1, 20000), _log(rng, 1, 20000)])
        form = rng.choice(["e4m3", "e4m3", "e2m1"])
        t = _log(rng, 1, 4096)
        if op == "norm":
            # 8-bit codes: a case of 4-bit ones would have to be unpacked for its output
            c = dict(op=op, n=rng.choice([1024, 2048, 4096, 5120, 7168, 8192, 32 * _log(rng, 1, 300)]), tokens=t,
                     post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]),
                     kind=rng.choice(["rms", "rms", "layer"]), scale=rng.choice([1.0, 0.25]), format="e4m3")
        elif op == "quantize":
            c = dict(op=op, t=t, k=rng.choice([k, 32 * _log(rng, 1, 500)]), swiglu=rng.random() < 0.5,
                     strided=rng.random() < 0.5, format="e4m3")
        elif op == "linear":
            c = dict(op=op, t=t, k=k, n=n, format=form)
        elif op == "swiglu":
            c = dict(op=op, t=t, k=k, inter=rng.choice([EXPERT, 1536, 5120, INTER, 32 * _log(rng, 1, 400)]), format=form,
                     to="e4m3")
        else:
            c = dict(op=op, t=t, k=k, inter=rng.choice([EXPERT, 1536, 5120, 128 * _log(rng, 1, 64)]), format=form)
        if _cost(c) <= top[op]:
            return c


def _width(form):
    """Bytes of a value in codes and scales."""
    return (1.0 if form == "e4m3" else 0.5) + 1 / 32


def _product(t, k, n):
    return n * k * 17 / 32, 2.0 * t * n * k


def work(c):
    op = c["op"]
    if op == "norm":
        e = float(c["tokens"]) * c["n"]
        read = 6 if c["gate"] == "token" else 4
        return {"bytes": e * (read + 2 + _width(c["format"])) + 2.0 * c["n"] * (1 + c["post"] + (c["gate"] == "channel")),
                "flops": e * 16}
    t, k = c["t"], c["k"]
    if op == "quantize":
        e = float(t) * k
        return {"bytes": e * ((4 if c["swiglu"] else 2) + _width(c["format"])), "flops": e * (12 if c["swiglu"] else 4)}
    if op == "linear":
        w, f = _product(t, k, c["n"])
        return {"bytes": w + t * k * _width(c["format"]) + 2.0 * t * c["n"], "flops": f}
    w, f = _product(t, k, 2 * c["inter"])
    if op == "swiglu":
        return {"bytes": w + t * k * _width(c["format"]) + t * c["inter"] * _width(c["to"]), "flops": f}
    w2, f2 = _product(t, c["inter"], k)
    return {"bytes": w + w2 + 8.0 * t * k, "flops": f + f2 + 16.0 * t * k}  # x, residual, r, y


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 250)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def _activations(g, t, n):
    """Rows as a decoder has them: some channels far larger than the rest."""
    channel = torch.exp(0.7 * _normal(g, n, dtype=torch.float32))
    return (_normal(g, t, n).float() * channel).to(torch.bfloat16)


def _nearest_e2m1(a):
    """Codes of magnitudes: the nearest of GRID, ties to the even code."""
    code = (a > 0.25).to(torch.uint8)
    for i, mid in enumerate((0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a >= mid) if i % 2 == 0 else (a > mid)
    return code


def _pack(z):
    """float32 values in the units of their blocks -> two E2M1 codes a byte, the even index low."""
    code = _nearest_e2m1(z.abs()) | (torch.signbit(z).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _weights(g, n, k):
    """MXFP4 weights as the library's packer makes them: the block's scale is floor(log2(largest)) - 2, values saturate."""
    q = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((n, k // 32), dtype=torch.uint8, device="cuda")
    for i in range(0, n, 16384):
        w = _normal(g, min(16384, n - i), k // 32, 32, dtype=torch.float32) * k ** -0.5
        e = torch.frexp(w.abs().amax(-1)).exponent - 3
        q[i:i + 16384] = _pack(torch.ldexp(w, -e[..., None]).clamp(-6, 6).flatten(1))
        s[i:i + 16384] = (e + 127).to(torch.uint8)
    return q, s


def _to_mx(z, form):
    """float32 [t, k] -> codes in units of their scales (E4M3 values, or packed E2M1) and E8M0 bytes."""
    b = z.unflatten(1, (-1, 32))
    m = torch.frexp(b.abs().amax(-1))
    if form == "e4m3":  # 448 is 0.875 * 2^9
        e = m.exponent - 9 + (m.mantissa > 0.875)
    else:  # 6 is 0.75 * 2^3
        e = m.exponent - 3 + (m.mantissa > 0.75)
    e = torch.where(m.mantissa == 0, -127, e).clamp(min=-127)
    b = torch.ldexp(b, -e[..., None]).flatten(1)
    return b.to(torch.float8_e4m3fn) if form == "e4m3" else _pack(b), (e + 127).to(torch.uint8)


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    s = {"case": c}
    op = c["op"]
    if op == "norm":
        t, n = c["tokens"], c["n"]
        s.update(x=_normal(g, t, n), residual=_activations(g, t, n), weight=_normal(g, n) * 0.1 + 1,
                 post=_normal(g, n) * 0.1 + 1 if c["post"] else None,
                 gate={"none": None, "channel": _normal(g, n), "token": _normal(g, t, n)}[c["gate"]],
                 bias=_normal(g, n) * 0.1 if c["kind"] == "layer" else None)
        return s
    t, k = c["t"], c["k"]
    if op == "quantize":
        width = 2 * k if c["swiglu"] else k
        x = _activations(g, t, width + 64 if c["strided"] else width)
        s["x"] = x[:, :width]
        return s
    if op == "block":
        s.update(x=_normal(g, t, k), residual=_activations(g, t, k), weight=_normal(g, k) * 0.1 + 1)
        s["w1"], s["w2"] = _weights(g, 2 * c["inter"], k), _weights(g, k, c["inter"])
        return s
    s["x"] = _to_mx(_activations(g, t, k).float(), c["format"])
    s["w"] = _weights(g, c["n"] if op == "linear" else 2 * c["inter"], k)
    return s


# ------------------------------------------------------------------- passes
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _codes(q, s):
    """8-bit codes and scales as the numbers that they are."""
    return {"codes": q, "scales": s.view(torch.float8_e8m0fnu)}


def _own_norm(s):
    import mxfp4_weight_streaming_gb300 as mx
    c = s["case"]
    q, scales, r = mx.residual_norm_mx(s["x"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"],
                                       bias=s["bias"], scale=c["scale"], kind=c["kind"], format=c["format"])
    return dict(_codes(q, scales), residual=r)


def _own_quantize(s):
    import mxfp4_weight_streaming_gb300 as mx
    return _codes(*mx.quantize_mx(s["x"], format=s["case"]["format"], swiglu=s["case"]["swiglu"]))


def _own_linear(s):
    import mxfp4_weight_streaming_gb300 as mx
    return mx.linear_mx(*s["x"], *s["w"])


def _own_swiglu(s):
    import mxfp4_weight_streaming_gb300 as mx
    return _codes(*mx.swiglu_mx(*s["x"], *s["w"], format=s["case"]["to"]))


def _own_block(s):
    import mxfp4_weight_streaming_gb300 as mx
    form = s["case"]["format"]
    q, scales, r = mx.residual_norm_mx(s["x"], s["residual"], s["weight"], format=form)
    h = mx.swiglu_mx(q, scales, *s["w1"], format=form)
    return {"y": mx.linear_mx(*h, *s["w2"]), "residual": r}


_own = {"norm": _own_norm, "quantize": _own_quantize, "linear": _own_linear, "swiglu": _own_swiglu, "block": _own_block}


def _values(q, s):
    """float32 values of codes (E4M3 or packed E2M1) and scales."""
    if q.dtype == torch.uint8:
        grid = torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")
        q = torch.stack((grid[(q & 15).int()], grid[(q >> 4).int()]), -1).flatten(1)
    e = s.to(torch.int32) - 127
    return torch.ldexp(q.float().unflatten(1, (-1, 32)), e[..., None]).flatten(1)


def _unit(x, kind, eps=1e-6):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def _norm32(s, kind="rms", scale=1.0):
    u = s["x"].float()
    if s.get("post") is not None:
        u = _unit(u, kind) * s["post"].float()
    if s.get("gate") is not None:
        u = u * s["gate"].float()
    r = s["residual"].float() + scale * u
    y = _unit(r, kind) * s["weight"].float()
    return (y if s.get("bias") is None else y + s["bias"].float()), r.to(torch.bfloat16)


def _silu(a):
    return a / (1 + torch.exp(-a))


def _plain_norm(s):
    c = s["case"]
    y, r = _norm32(s, c["kind"], c["scale"])
    return dict(_codes(*_to_mx(y, c["format"])), residual=r)


def _plain_quantize(s):
    z = s["x"].float()
    if s["case"]["swiglu"]:
        k = s["case"]["k"]
        z = _silu(z[:, :k]) * z[:, k:]
    return _codes(*_to_mx(z, s["case"]["format"]))


def _dot(x, w):
    return _values(*x) @ _values(*w).T


def _plain_linear(s):
    return _dot(s["x"], s["w"]).to(torch.bfloat16)


def _gated(x, w, form):
    ab = _dot(x, w)
    inter = ab.shape[1] // 2
    return _to_mx(_silu(ab[:, :inter]) * ab[:, inter:], form)


def _plain_swiglu(s):
    return _codes(*_gated(s["x"], s["w"], s["case"]["to"]))


def _plain_block(s):
    form = s["case"]["format"]
    y, r = _norm32(s)
    h = _gated(_to_mx(y, form), s["w1"], form)
    return {"y": _dot(h, s["w2"]).to(torch.bfloat16), "residual": r}


_plain = {"norm": _plain_norm, "quantize": _plain_quantize, "linear": _plain_linear, "swiglu": _plain_swiglu,
          "block": _plain_block}


# ------------------------------------------------------- definitions, 64 bits
def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits. Codes are given as the unrounded quotients that they stand
    for; a block's scale is a choice between powers of two and has no value to be near to: None."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        y, r = _exact_norm(s, c["kind"], c["scale"])
        return {"codes": _exact_blocks(y, c["format"])[0], "scales": None, "residual": r}
    if c["op"] == "quantize":
        z = s["x"].double()
        if c["swiglu"]:
            z = z[:, :c["k"]] * torch.sigmoid(z[:, :c["k"]]) * z[:, c["k"]:]
        return {"codes": _exact_blocks(z, c["format"])[0], "scales": None}
    if c["op"] == "linear":
        return _exact_dot(*_exact_codes(s["x"]), s["w"])
    if c["op"] == "swiglu":
        return {"codes": _exact_blocks(_exact_gated(*_exact_codes(s["x"]), s["w"]), c["to"])[0], "scales": None}
    y, r = _exact_norm(s, "rms", 1.0)
    h = _exact_gated(*_exact_rounded(y, c["format"]), s["w1"])
    return {"y": _exact_dot(*_exact_rounded(h, c["format"]), s["w2"]), "residual": r}


def _exact_norm(s, kind, scale):
    def normed(z):
        mean = z.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(z[:, :1])
        return (z - mean) / torch.sqrt((z - mean).pow(2).mean(1, keepdim=True) + 1e-6)

    u = s["x"].double()
    if s.get("post") is not None:
        u = normed(u) * s["post"].double()
    if s.get("gate") is not None:
        u = s["gate"].double() * u
    r = s["residual"].double() + u * scale
    y = normed(r) * s["weight"].double()
    return (y + s["bias"].double() if s.get("bias") is not None else y), r


def _exact_blocks(z, form):
    """(values / 2^e, e) of the blocks: e the least integer that keeps every |value| / 2^e within the type."""
    b = z.view(z.shape[0], -1, 32)
    e = torch.ceil(torch.log2(b.abs().amax(2) / MOST[form])).clamp(min=-127)
    return (b / torch.exp2(e)[:, :, None]).view(z.shape), e


def _exact_rounded(z, form):
    """Blocks rounded to their type's points, nearest and ties to even, as float64 values and exponents."""
    v, e = _exact_blocks(z, form)
    low, bits = (-6, 3) if form == "e4m3" else (0, 1)  # least normal exponent, bits of the fraction
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))) - bits)
    return torch.round(v / step) * step, e


def _exact_codes(x):
    q, s = x
    if q.dtype == torch.uint8:
        codes = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.uint8, device="cuda")
        codes[:, ::2], codes[:, 1::2] = q % 16, q // 16
        m = codes % 8
        q = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5) * torch.exp2(m // 2 - 1.0)) * torch.where(codes > 7, -1.0, 1.0)
    return q.double(), s.double() - 127


def _exact_dot(v, e, w):
    """Sum over the blocks of 2^(e + f) times the blocks' dot products, summed in 64 bits. A block's 32 products of codes
    are whole multiples of a power of two; taken apart into values of at least 1/4 and below, their sums fit the 24 bits
    of a float32, whose products are far faster and lose nothing."""
    wv, f = _exact_codes(w)
    out = torch.zeros((v.shape[0], wv.shape[0]), dtype=torch.float64, device="cuda")
    large = torch.where(v.abs() >= 0.25, v, 0.0)
    for part in (large, v - large):
        if not bool(part.any()):
            continue
        for b in range(e.shape[1]):
            at = slice(32 * b, 32 * b + 32)
            dots = part[:, at].float() @ wv[:, at].float().T
            scale = torch.exp2(f[:, b])
            for i in range(0, out.shape[0], 1024):
                out[i:i + 1024].addcmul_(dots[i:i + 1024] * torch.exp2(e[i:i + 1024, b, None]), scale)
    return out


def _exact_gated(v, e, w):
    ab = _exact_dot(v, e, w)
    a, b = ab.chunk(2, 1)
    return a * torch.sigmoid(a) * b
