"""Shared helpers for the tests of microscaled activations and their products:
the codes' values and the operators' definitions in float64."""
from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MOST = {"e4m3": 448.0, "e2m1": 6.0}
# Bits of the fraction and the least normal exponent of the element types.
FRACTION = {"e4m3": (3, -6), "e2m1": (1, 0)}


def elements(q):
    """float64 elements of codes: float8 values, or packed E2M1."""
    if q.dtype == E4M3:
        return q.double()
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=q.device)
    return torch.stack((grid[(q & 15).long()], grid[(q >> 4).long()]), -1).flatten(1)


def power(s):
    """2 ** (byte - 127) in float64; 255 is NaN."""
    return torch.where(s == 255, torch.nan, torch.exp2(s.double() - 127))


def values(q, s):
    return elements(q) * power(s).repeat_interleave(32, 1)


def round_to(z, form):
    """float64 elements (within the type's range) rounded to nearest, ties to even."""
    bits, low = FRACTION[form]
    e = torch.frexp(z)[1].double() - 1
    step = torch.exp2(torch.where(z == 0, float(low), e).clamp(min=low) - bits)
    return torch.round(z / step) * step


def scale_exponents(z, form):
    """Least e >= -127 with max|z| <= most * 2^e, per block of 32 of float64 rows."""
    top = z.unflatten(1, (-1, 32)).abs().amax(-1)
    m, p = torch.frexp(top)  # most = 0.875 * 2^9 or 0.75 * 2^3
    e = p - 9 + (m > 0.875) if form == "e4m3" else p - 3 + (m > 0.75)
    return torch.where(top == 0, -127, e).clamp(min=-127)


def check_codes(q, s, z, form, slack, what):
    """Codes and scales of float64 z that was computed in fp32, off by up to
    slack (a tensor) at most: a scale is the least that fits, up to the slack at the
    border; a value is off by half a step of its type and the slack."""
    e = s.double() - 127
    top = z.unflatten(1, (-1, 32)).abs().amax(-1)
    room = slack.unflatten(1, (-1, 32)).amax(-1)
    assert (s != 255).all(), f"{what}: NaN scales"
    assert (top - room <= MOST[form] * torch.exp2(e)).all(), f"{what}: a scale is too small"
    assert ((top + room > MOST[form] * torch.exp2(e - 1)) | (s == 0)).all(), f"{what}: a scale is too large"
    bits, low = FRACTION[form]
    unit = torch.exp2(e).repeat_interleave(32, 1)
    half = torch.maximum(z.abs() * 2.0 ** -(bits + 1), unit * 2.0 ** (low - bits - 1))
    off = (values(q, s) - z).abs()
    bad = off > half + slack * (1 + 2.0 ** -bits)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: "
                             f"{float(values(q, s)[i])} for {float(z[i])}")


def random_codes(g, t, k, form, spread=5):
    """Any element of the type but NaN, scales of 2^-spread to 2^spread."""
    s = torch.randint(127 - spread, 128 + spread, (t, k // 32), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    if form == "e2m1":
        return torch.randint(0, 256, (t, k // 2), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8), s
    q = torch.randint(0, 254, (t, k), generator=g, device="cuda", dtype=torch.int32)
    q = q + (q >= 127).int()  # 0x7f and 0xff are NaN
    return q.to(torch.uint8).view(E4M3), s


def product(x, w):
    """(sum_k x w, sum_k |x w|) in float64 of (codes, scales) pairs."""
    a, b = values(*x), values(*w)
    return a @ b.T, a.abs() @ b.abs().T


def sum_bound(k, mag):
    """Error of a sum over k in the tensor cores. An instruction adds 32 (E2M1: 64)
    exact products and the running sum, each cut to the 24 bits of an fp32 number
    of the largest of them at worst: 2^-23 of it, which is at most sum |x w|, for the
    products' sum and for the running sum, k / 32 times."""
    return 2 * (k / 32 + 1) * 2.0 ** -23 * mag
