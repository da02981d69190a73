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


@pytest.mark.parametrize("default", [False, True], ids=["side", "default"])
def test_a_dropped_plane_of_quantize_act(default):
    """quantize_act and the product on one handle, the plane dropped once both are enqueued: the current stream
    must not be handed its memory while they run."""
    import torch
    from block_quantized_matmul_mq_amd import mq
    c = Calls(seed=6)
    ref = c.gemm_ep()[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    on, current = (torch.cuda.default_stream(), side) if default else (side, torch.cuda.default_stream())
    size = c.Xq.numel()
    for turn in range(10):
        say(f"quantize_act and gemm_ep on handle {on.cuda_stream}, turn {turn}")
        with torch.cuda.stream(on):
            keep_busy(c.X.device)
        with torch.cuda.stream(current):
            Xq = mq.quantize_act(c.Xg, stream=on.cuda_stream)
            out = mq.gemm_ep(c.W, mq.Q4_K, Xq, 40, c.N, c.X.shape[1], act=mq.ACT_SILU, mul=c.mulg, stream=on.cuda_stream)
            del Xq
            for _ in range(4):
                torch.full((size,), 255, dtype=torch.uint8, device=c.X.device)
        torch.cuda.synchronize()
        assert torch.equal(out, ref), turn
