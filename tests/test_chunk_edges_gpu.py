"""The calls for many tokens as programs make them: captured and replayed, on
several streams at once, into the caller's memory, with sizes past 2^31, and
waits that run out."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from chunk_cases import E4M3, elements, product, random_codes, sum_bound, values
from gpu_cases import Guarded, lib
from step_cases import check, gen, randn

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bits(t):
    return t.view(U8) if t.dtype == E4M3 else t.view(torch.int16) if t.dtype == BF16 else t


def same(a, b):
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


class Block:
    """An FFN block's weights, and its calls."""

    def __init__(self, seed, k=512, inter=640):
        mx, g = lib(), gen(seed)
        self.norm = randn(g, k) * 0.1 + 1
        self.w1 = mx.quantize(torch.randn(2 * inter, k, generator=g, device="cuda") * k ** -0.5)
        self.w2 = mx.quantize(torch.randn(k, inter, generator=g, device="cuda") * inter ** -0.5)

    def __call__(self, x, res, form, stream=None):
        mx = lib()
        q, s, r = mx.residual_norm_mx(x, res, self.norm, format=form, stream=stream)
        h = mx.swiglu_mx(q, s, *self.w1, format=form, stream=stream)
        return mx.linear_mx(*h, *self.w2, stream=stream), r


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
@pytest.mark.parametrize("t", [1, 40, 300])
def test_captured_and_replayed(form, t):
    """The first calls of these sizes are made in the capture; replays read what the inputs hold by then."""
    g = gen(t)
    block = Block(3)
    x, res = randn(g, t, 512), randn(g, t, 512)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, r = block(x, res, form)
        y, r = block(y, r, form)
    for _ in range(3):
        x.copy_(randn(g, t, 512))
        res.copy_(randn(g, t, 512))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), r.clone()
        assert same(got, block(*block(x, res, form), form))


def test_streams_at_once():
    """Two streams run blocks of their own next to each other; each result is the one that a stream alone gives."""
    mx, g = lib(), gen(9)
    blocks = [Block(1), Block(2, inter=1024)]
    xs = [(randn(g, t, 512), randn(g, t, 512)) for t in (50, 700)]
    alone = [b(*x, "e4m3") for b, x in zip(blocks, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            got[i].append(blocks[i](*xs[i], "e4m3", stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for one in got[i]:
            assert same(one, alone[i])
    assert mx.last_device_status() == mx.MXFP4_OK


def test_weights_made_just_before():
    """Codes of quantize_mx are weights too, in the very next call; older ones must not be what is read."""
    mx, g = lib(), gen(10)
    x = mx.quantize_mx(randn(g, 130, 1024), "e2m1")
    q, s = torch.empty(512, 512, dtype=U8, device="cuda"), torch.empty(512, 32, dtype=U8, device="cuda")
    for form in ("e2m1", "e4m3"):
        a = x if form == "e2m1" else mx.quantize_mx(randn(g, 130, 1024), "e4m3")
        got, want = [], []
        ws = [randn(g, 512, 1024) for _ in range(6)]
        for w in ws:
            mx.quantize_mx(w, "e2m1", out=(q, s))
            got.append(mx.linear_mx(*a, q, s))
        for w in ws:
            m = mx.quantize_mx(w, "e2m1")
            torch.cuda.synchronize()
            want.append(mx.linear_mx(*a, *m))
            torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_same_bits_every_time(form):
    mx, g = lib(), gen(11)
    for t, n, k in ((3, 700, 4096), (200, 300, 2048), (600, 1000, 1024)):
        x, w = random_codes(g, t, k, form), random_codes(g, n, k, "e2m1")
        first = mx.linear_mx(*x, *w)
        for _ in range(5):
            assert torch.equal(bits(mx.linear_mx(*x, *w)), bits(first))


@pytest.mark.parametrize("n", [33, 64, 129, 136, 1000, 1007])
@pytest.mark.parametrize("t", [1, 70, 300])
def test_rows_of_y_at_any_even_address(t, n):
    mx, g = lib(), gen(t + n)
    k = 384
    x, w = random_codes(g, t, k, "e4m3"), random_codes(g, n, k, "e2m1")
    ref, mag = product(x, w)
    whole = Guarded((t * n + 8,), BF16)
    for off in (1, 3, 4):
        whole.t.fill_(7.0)
        y = whole.t[off:off + t * n].view(t, n)
        mx.linear_mx(*x, *w, out=y)
        whole.check("y")
        assert (whole.t[:off] == 7).all() and (whole.t[off + t * n:] == 7).all()
        check(y, ref, ref.abs() * 2.0 ** -8 + sum_bound(k, mag), f"offset {off}")


def test_scales_at_any_word():
    """Weights of one expert among many: scales that begin at any multiple of 4 bytes."""
    mx, g = lib(), gen(13)
    k, n = 1024, 96
    wq, ws = random_codes(g, 4 * n, k, "e2m1")
    x = random_codes(g, 20, k, "e4m3")
    flat = torch.empty(ws.numel() + 64, dtype=U8, device="cuda")
    for off in (4, 8, 12):
        moved = flat[off:off + ws.numel()].view_as(ws).copy_(ws)
        for i in range(4):
            rows = slice(i * n, (i + 1) * n)
            got = mx.linear_mx(*x, wq[rows], moved[rows])
            assert torch.equal(bits(got), bits(mx.linear_mx(*x, wq[rows].clone(), ws[rows].clone())))


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_outputs_past_2_31(form):
    """More than 2^31 outputs: places in y are counted in 64 bits."""
    mx, g = lib(), gen(14)
    t, n, k = 70000, 33000, 128
    x, w = random_codes(g, t, k, form), random_codes(g, n, k, "e2m1")
    y = mx.linear_mx(*x, *w)
    for rows in (slice(0, 3), slice(34990, 35010), slice(65070, 65090), slice(t - 3, t)):
        ref, mag = product((x[0][rows], x[1][rows]), w)
        check(y[rows], ref, ref.abs() * 2.0 ** -8 + sum_bound(k, mag), f"rows {rows}")


def test_weights_past_2_31():
    """More than 2^31 bytes of weight codes."""
    mx, g = lib(), gen(15)
    n, k = 600000, 7168
    x = random_codes(g, 2, k, "e4m3")
    wq = torch.empty(n, k // 2, dtype=U8, device="cuda")
    wq.view(torch.int32).random_(generator=g)
    ws = torch.randint(122, 132, (n, k // 32), generator=g, device="cuda", dtype=torch.int32).to(U8)
    y = mx.linear_mx(*x, wq, ws)
    for rows in (slice(0, 300), slice(599000, 599300), slice(n - 5, n)):
        ref, mag = product(x, (wq[rows], ws[rows]))
        check(y[:, rows], ref, ref.abs() * 2.0 ** -8 + sum_bound(k, mag), f"rows {rows}")


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_the_longest_k(form):
    """k of 2^24, all but a few values 0: their sums are exact in fp32, so only the rounding to bf16 is left."""
    mx, g = lib(), gen(19)
    k = 1 << 24
    x, w = torch.zeros(3, k, dtype=BF16, device="cuda"), random_codes(g, 5, k, "e2m1", spread=1)
    at = torch.tensor([0, 5, 4097, k // 2 + 3, k - 129, k - 1], device="cuda")
    x[:, at] = torch.tensor([[1.0, 2, 4, 1, 2, 1], [0, 0, 0, 0, 0, 1], [1, 0, 0, -4, 0, 0]], device="cuda").to(BF16)
    y = mx.linear_mx(*mx.quantize_mx(x, form), *w)
    assert mx.last_device_status() == mx.MXFP4_OK
    ref = x[:, at].double() @ values(*w)[:, at].T
    assert torch.equal(y, ref.to(BF16))


def test_quantize_past_2_31():
    mx, g = lib(), gen(16)
    x = torch.empty(300000, 8192, dtype=BF16, device="cuda")
    x.fill_(1.0)
    x[-2:] = randn(g, 2, 8192)
    q, s = mx.quantize_mx(x)
    ref = mx.quantize_mx(x[-2:].clone())
    assert torch.equal(bits(q[-2:]), bits(ref[0])) and torch.equal(s[-2:], ref[1])
    assert (q[:2].float() == 256).all() and (s[:2] == 119).all()
    assert elements(q[150000:150001]).eq(256).all()


def test_on_the_hosts_terms():
    """stream= with the caller's memory, and an empty batch."""
    mx, g = lib(), gen(17)
    x, w = randn(g, 9, 256), random_codes(g, 64, 256, "e2m1")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = mx.quantize_mx(x)
    y = torch.zeros(9, 64, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    q = (torch.zeros_like(out[0]), torch.zeros_like(out[1]))
    side.wait_stream(torch.cuda.current_stream())
    assert mx.quantize_mx(x, out=q, stream=side) == q
    assert mx.linear_mx(*q, *w, out=y, stream=side) is y
    torch.cuda.synchronize()
    assert same(q, out) and torch.equal(bits(y), bits(mx.linear_mx(*out, *w)))
    for call in (lambda: mx.quantize_mx(x[:0]), lambda: mx.linear_mx(out[0][:0], out[1][:0], *w)):
        with pytest.raises(mx.Mxfp4Error):
            call()
    with pytest.raises(mx.Mxfp4Error):
        mx.linear_mx(*mx.quantize_mx(randn(g, 2, 96)), *random_codes(g, 64, 96, "e2m1"))  # k


@pytest.fixture(scope="module")
def withhold_lib():
    """The test-only build of test_timeout_gpu.py: CTA 0 never gets its first stage, waits end after 1 ms."""
    from mxfp4_weight_streaming_gb300 import build
    path = build.build_test_variant("withhold", ["MXFP4_TEST_WITHHOLD_STAGE", "MXFP4_WAIT_LIMIT_NS=1000000ull"])
    L = ctypes.CDLL(path)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.mxfp4_linear_mx.restype = I
    L.mxfp4_linear_mx.argtypes = [P, P, I, I64, I64, P, P, I64, P, P]
    L.mxfp4_last_device_status.restype = I
    L.mxfp4_last_device_status.argtypes = [P]
    return L


# One CTA a tile; a cluster that shares one; pairs, with many tiles each.
@pytest.mark.parametrize("t,n,k", [(100, 20000, 256), (16, 1024, 7168), (1000, 20000, 512)])
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_waits_run_out(withhold_lib, t, n, k, form):
    mx, g = lib(), gen(18)
    x, w = random_codes(g, t, k, form), random_codes(g, n, k, "e2m1")
    y = torch.zeros(t, n, dtype=BF16, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert mx.last_device_status() == mx.MXFP4_OK
    rc = withhold_lib.mxfp4_linear_mx(x[0].data_ptr(), x[1].data_ptr(), 0 if form == "e4m3" else 1, t, k, w[0].data_ptr(),
                                      w[1].data_ptr(), n, y.data_ptr(), stream)
    assert rc == mx.MXFP4_OK  # the launch itself succeeds
    assert withhold_lib.mxfp4_last_device_status(stream) == mx.MXFP4_ERR_TIMEOUT
    assert withhold_lib.mxfp4_last_device_status(stream) == mx.MXFP4_OK  # read and cleared
    mx.linear_mx(*x, *w, out=y)
    ref, mag = product(x, w)
    check(y, ref, ref.abs() * 2.0 ** -8 + sum_bound(k, mag), "afterwards")
    assert values(*w).isfinite().all()


# ---------------------------------------------------------------- example
@pytest.fixture(scope="module")
def ex():
    lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import verify_step
    return verify_step


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_prompt_in_chunks(ex, form):
    """A prompt in one chunk, twice, and in three: the same bits, and what eight
    quantisations in a row (two layers) may make of other orders of the sums: each
    rounds by at most 2^-4 (2^-2) of its input."""
    model = ex.Decoder(layers=2, hidden=512, heads=4, kv_heads=2, inter=512, vocab=512)
    tokens = torch.arange(300, device="cuda") * 11 % 512
    rows = []
    for sizes in ([300], [300], [100, 37, 163]):
        seq, out, at = ex.Sequences(model.new_cache(64), 1, 32), [], 0
        for n in sizes:
            seq.room(n)
            out.append(model.prompt_chunk(tokens[at:at + n], seq.cache, seq.batch(n, 512), form))
            at += n
        rows.append(torch.cat(out))
        assert int(seq.lens) == 300
    assert torch.equal(bits(rows[0]), bits(rows[1]))
    a, b = rows[0].double(), rows[2].double()
    assert a.isfinite().all() and (a - b).norm() < 8 * (2 ** -4 if form == "e4m3" else 2 ** -2) * a.norm()


def test_example_with_a_long_prompt():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "verify_step.py"), "--layers", "1", "--steps", "3",
                        "--prompt", "700", "--prompt-chunk", "256"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "verify steps" in r.stdout
