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


@pytest.mark.parametrize("default", [False, True], ids=["side", "default"])
@pytest.mark.parametrize("name", ["gemv", "gemm", "repack", "gemm_blockdots"])
def test_products_without_buffers(name, default):
    """The products' own outputs and workspaces (a K that is cut) on a handle while another stream is busy."""
    import torch
    from block_quantized_matmul_mq_amd import mq
    from gpu_cases import device, to_dev, weights
    dev = device()
    M, N, K = 40, 100, 8192
    W = to_dev(weights(mq.Q4_K, N, K, "random", 41).reshape(-1), dev)
    X = torch.randn(M, K, device=dev)
    Xq, x = mq.quantize_act(X), X[0].contiguous()
    assert mq.gemm_scratch_bytes(mq.Q4_K, M, N, K) > 0
    call = {"gemv": lambda **k: mq.gemv(W, mq.Q4_K, x, N, K, **k), "gemm": lambda **k: mq.gemm(W, mq.Q4_K, Xq, M, N, K, **k),
            "repack": lambda **k: mq.repack(W, mq.Q4_K, N, K, **k),
            "gemm_blockdots": lambda **k: mq.gemm_blockdots(W, mq.Q4_K, Xq, M, N, K, **k)}[name]
    ref = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    on, current = (torch.cuda.default_stream(), side) if default else (side, torch.cuda.default_stream())
    for turn in range(5):
        say(f"{name} on handle {on.cuda_stream}, turn {turn}")
        with torch.cuda.stream(current):
            keep_busy(dev)
            out = call(stream=on.cuda_stream)
        on.synchronize()
        assert torch.equal(out.cpu(), ref.cpu()), turn
        torch.cuda.synchronize()
