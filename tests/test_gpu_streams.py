"""Calls on a stream handle that is not the current stream's: what the binding makes belongs to that stream."""

import pytest

from gpu_cases import say
from test_gpu_ffn_calls import NAMES, Calls

pytestmark = pytest.mark.gpu


def keep_busy(dev):
    """Work on the current stream, whose freed memory then holds other values."""
    import torch
    x = torch.randn(4096, 4096, device=dev)
    for _ in range(4):
        x = (x @ x).clamp_(-1, 1)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=dev) for _ in range(4)]
    del junk


@pytest.mark.parametrize("M", [1, 5])
@pytest.mark.parametrize("name", NAMES)
def test_the_default_streams_handle(name, M):
    """Handle 0 while another stream is current."""
    import torch
    c = Calls(M, seed=5)
    ref = getattr(c, name)()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for turn in range(5):
        say(f"{name} M={M} on handle 0, call {turn}")
        with torch.cuda.stream(side):
            keep_busy(c.X.device)
            out = getattr(c, name)(stream=0)
        torch.cuda.default_stream().synchronize()
        for a, b in zip(ref, out):
            assert torch.equal(a.cpu(), b.cpu()), turn
        torch.cuda.synchronize()
