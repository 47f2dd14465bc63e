"""The step's norms, rotary positions and page bookkeeping where calls go to
their limits."""
import pytest
import torch

from gpu_cases import lib
from step_cases import gen, randn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


# ------------------------------------------------------------------- streams
def test_results_on_another_stream_are_not_memory_of_the_current_ones_work():
    """The current stream still has to write into memory that the host has given back; a call on another stream,
    which does not wait for that, may not be handed it."""
    mx = lib()
    g = gen(1)
    x, res, w = randn(g, 64, 4096), randn(g, 64, 4096), randn(g, 4096)
    y0, r0 = mx.residual_norm(x, res, w)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    late = [torch.empty_like(x).fill_(7) for _ in range(2)]
    del late
    y, r = mx.residual_norm(x, res, w, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(r, r0)
